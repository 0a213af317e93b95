"""Loss scales near the end of fp32 (a dynamic scale over fp32 or bf16 gradients
grows until they overflow, up to 2^127): unscaling and clipping keep their
precision where the product of the two factors is below fp32's normal numbers."""
import numpy as np
import pytest
import torch

from test_gpu_multi_list import HP, check_step, lay_out, make, snapshot, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    assert torch.cuda.is_available()
    return m


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [[700, 5, 2049], [64] * 2100], ids=["short", "long"])
@pytest.mark.parametrize("log2_scale,max_norm", [(110, 1e-6), (120, 1e-8), (126, 1e-3), (126, 1.0)])
def test_scale_near_the_end_of_fp32(zf, n, dtype, bits, log2_scale, max_norm):
    """The same bounds as at any other scale."""
    scale = 2.0 ** log2_scale
    hp = dict(HP, max_grad_norm=max_norm, eps=1e-12)
    opt, ref, (_, copies) = make(zf, n, bits, dtype, torch.bfloat16, "packed", scale, hp=hp)
    for t in (1, 2):
        # unscaled gradients below 2: their scaled values stay below fp32's largest
        vals = [np.clip(v, -1.9, 1.9) * scale for v in values(n, 40 + t, 0.3)]
        _, grads = lay_out(vals, "packed", dtype)
        opt.bind(grads, copies)
        before = snapshot(opt)
        opt.step()
        check_step(opt, ref, grads, before, t, scale, copies, bits)
