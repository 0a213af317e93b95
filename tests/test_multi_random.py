"""The numbers that second moments are rounded with, from their definition: what
seeds share, and that well-separated ones share nothing (no GPU needed)."""
import numpy as np
import pytest

from list_reference import random16


def test_the_next_seed_has_a_steps_numbers_a_step_earlier():
    assert np.array_equal(random16(16, 5, 7), random16(16, 4, 8))


@pytest.mark.parametrize("a,b", [((1, 0), (2, 0)), ((1, 0), (1, 1 << 20)), ((9, 1 << 20), (9, 1 << 21))])
def test_other_steps_and_distant_seeds_are_uncorrelated(a, b):
    """64 rows of 256: the correlation of N independent pairs has a spread of
    1/sqrt(N); their means are half the range within 6 of theirs."""
    x, y = (random16(64, *p).reshape(-1) for p in (a, b))
    n = x.size
    for z in (x, y):
        assert abs(z.mean() / 65536 - 0.5) <= 6 / np.sqrt(12 * n)
    assert abs(np.corrcoef(x, y)[0, 1]) <= 6 / np.sqrt(n)
    # equal numbers in one place: 1 in 65536 by chance
    assert np.sum(x == y) <= 6
