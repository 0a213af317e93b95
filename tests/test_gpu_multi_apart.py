"""Statistics of a list taken apart from its step: with other ranks' sums between
the two, on lists of every length, and as a look between steps."""
import math

import numpy as np
import pytest
import torch

from test_gpu_multi_list import HP, f64, lay_out, make, snapshot, values
from test_gpu_multi_list import SIZES as SHORT
from test_gpu_multi_long import SIZES as LONG
from test_gpu_multi_long import check_arenas

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    assert torch.cuda.is_available()
    return m


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("sizes", ["tiles", "large", "tensors"])
def test_a_step_with_other_ranks_sums(zf, sizes, apart, bits):
    """The clip covers this list's sum and the remote one, whether the step
    takes the statistics itself or finds them taken, as a rank does that
    exchanges them first."""
    n = SHORT.get(sizes) or LONG[sizes]
    opt, ref, (_, copies) = make(zf, n, bits, torch.float16, torch.bfloat16, "packed", 512.0)
    for t, remote in ((1, 0.0), (2, 700.0), (3, 5e6)):
        _, grads = lay_out(values(n, 30 + t, 0.5), "packed", torch.float16)
        opt.bind(grads, copies)
        before = snapshot(opt)
        if apart:
            zf.zero_multi_unscale_norm(opt.plan, opt.state)
            opt.state.field("remote_sumsq").copy_(torch.tensor(remote, device="cuda"))
            zf.zero_multi_adamw_step(opt.plan, opt.master, opt.exp_avg, opt.exp_avg_sq, opt.hp,
                                     opt.state, exp_avg_scale=opt.exp_avg_scale,
                                     exp_avg_sq_scale=opt.exp_avg_sq_scale, seed=opt.seed)
        else:
            opt.state.set_remote(remote)
            opt.step()
        mine = sum(float(np.sum((f64(g) / 512.0) ** 2)) for g in grads)
        norm = math.sqrt(mine + remote)
        st = opt.state.read()
        assert abs(st.last_norm - norm) <= 1e-10 * norm
        assert (st.step, st.last_skipped, st.remote_sumsq, st.sumsq) == (t, 0, remote, 0.0)
        coef = min(1.0, HP["max_grad_norm"] / (norm + 1e-6))
        assert abs(st.last_coef - coef) <= 2.0 ** -24 * coef * 1.001
        # the reference clips by its own gradients: the limit that gives this coefficient
        ref.hp = dict(HP, max_grad_norm=coef * (math.sqrt(mine) + 1e-6))
        check_arenas(ref, grads, before, snapshot(opt), t, 512.0, bits)
        for c, p in zip(copies, opt.views(opt.master)):
            assert torch.equal(c, p.to(c.dtype))
    opt.state.set_remote(0.0, 1)                           # another rank's overflow
    before = snapshot(opt)
    opt.step()
    assert opt.state.read().last_skipped == 1
    assert all(np.array_equal(a, b) for a, b in zip(snapshot(opt), before))


@pytest.mark.parametrize("sizes", ["spans", "tensors"])
def test_statistics_taken_between_steps(zf, sizes):
    """A look at the statistics takes a state of its own, or clears the step's
    two fields afterwards: what they hold is added to the next step's."""
    n = SHORT.get(sizes) or LONG[sizes]
    opt, _, (_, copies) = make(zf, n, 32, torch.bfloat16, torch.bfloat16, "own", 4.0)
    _, grads = lay_out(values(n, 9, 0.3), "own", torch.bfloat16)
    opt.bind(grads, copies)
    norm = math.sqrt(sum(float((g.double() / 4.0).square().sum()) for g in grads))
    look = zf.StepState(4.0, False)
    zf.zero_multi_unscale_norm(opt.plan, look, reset=True)
    assert abs(look.read().sumsq - norm ** 2) <= 1e-10 * norm ** 2
    opt.step()
    assert abs(opt.state.read().last_norm - norm) <= 1e-10 * norm
    zf.zero_multi_unscale_norm(opt.plan, opt.state, reset=True)
    opt.state.field("sumsq").zero_()
    opt.state.field("overflow").zero_()
    opt.step()
    assert abs(opt.state.read().last_norm - norm) <= 1e-10 * norm
    zf.zero_multi_unscale_norm(opt.plan, opt.state, reset=True)
    opt.step()
    assert abs(opt.state.read().last_norm - math.sqrt(2) * norm) <= 1e-10 * norm
