"""Which kernels the lists of the GPU tests reach, from the plan's own tables
(no GPU needed): moving a limit between variants must not leave one untested."""
import numpy as np
import pytest
import torch

import test_gpu_multi_list as short_lists
import test_gpu_multi_long as long_lists


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    return m


def tile_rows(zf, n):
    return zf.MultiPlan(n, torch.bfloat16, torch.bfloat16, 8, device="cpu")._plan.tile_rows


def test_every_tile_height_is_reached(zf):
    got = {name: tile_rows(zf, n) for name, n in short_lists.SIZES.items()}
    assert got == {"one": 1, "rows": 1, "tiles": 1, "spans": 1, "many": 1, "large": 2}
    assert {name: tile_rows(zf, n) for name, n in long_lists.SIZES.items()} == \
        {name: 4 for name in long_lists.SIZES}


def test_long_lists_reach_every_shift_and_end(zf):
    """Packed behind one element, the whole tiles of the long lists start at
    every element of an 8-byte word, and their last tiles have 1 to 4 rows."""
    for name in ("tensors", "elements"):
        n = np.array(long_lists.SIZES[name])
        first = 1 + np.concatenate(([0], np.cumsum(n)[:-1]))
        assert set(first[n >= 1024] % 4) == {0, 1, 2, 3}, name
    n = np.array(long_lists.SIZES["tensors"])
    assert set(-(-(n % 1024) // 256)) == {0, 1, 2, 3, 4}


def test_the_sliced_list_takes_two_launches(zf):
    plan = zf.MultiPlan([long_lists.SLICED], torch.bfloat16, torch.bfloat16, 8, device="cpu")._plan
    assert plan.tile_rows == 4 and 131072 < plan.n_tiles < 2 * 131072
