"""The embedding, the 8-bit activations and the weight gradients together, as a
rank's step uses them (examples/unit_saved8.py): the gradients in the flat buffer
against the chain rule in 64 bits over what the checkpoints stand for, the step
taken from them against the CPU oracle, an overflow in the activations that
skips the step, and the whole round captured in a graph."""
import math
import os
import sys

import numpy as np
import pytest
import torch

from harness import assert_bitwise, to_host

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
BF, F32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def ex():
    import unit_saved8
    assert torch.cuda.is_available()
    return unit_saved8


def batch_of(ex, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, ex.VOCAB, (n,), generator=g, device="cuda")
    t[: n // 4] = 17
    return t, torch.randint(0, ex.VOCAB, (n,), generator=g, device="cuda")


def values(s):
    table = torch.tensor([2.0 ** (e - 133) for e in range(255)] + [math.nan], dtype=torch.float64, device="cuda")
    x = s.codes.view(*s.exponents.shape, 32).double() * table[s.exponents.long()][:, :, None]
    return x.view(s.codes.shape)[:, :s.cols]


def near(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), got[bad][:3], want[bad][:3], tol.expand_as(want)[bad][:3])


def test_gradients_in_the_flat_buffer(ex):
    n = 300
    unit = ex.Unit(n)
    tokens, targets = batch_of(ex, n, 3)
    unit.gather()
    logits = unit.forward(tokens)
    _, d = ex.loss_and_gradient(logits, targets, 1024.0)
    unit.grad.fill_(7.0)
    unit.backward(tokens, d)
    torch.cuda.synchronize()
    w = [x.double() for x in unit.weights]
    s = {k: values(v) for k, v in unit.saved.items()}

    def mm(a, b):
        return torch.matmul(a.contiguous(), b.contiguous())

    # each product's sums are fp32 (k additions) and its result one rounding to bf16
    def product(a, b, off=0.0):
        y, size = mm(a, b), mm(a.abs(), b.abs())
        tol = size * a.shape[1] * 2 * F32 + (mm(off, b.abs()) if torch.is_tensor(off) else 0.0)
        return y, tol + (y.abs() + tol) * BF

    d16 = d.bfloat16().double()
    head = mm(d16.t(), s["y"])
    near(unit.grads[3], head, mm(d16.abs().t(), s["y"].abs()) * n * 2 * F32)
    dy, dy_tol = product(d16, w[3])
    dh, dh_tol = product(dy, w[2], dy_tol)
    gate, up = s["gate"], s["up"]
    sig = torch.sigmoid(gate)
    act, slope = gate * sig, sig * (1 + gate * torch.sigmoid(-gate))
    # the output's checkpoint made anew, within a code of it (half, or one where it was cut at 127)
    unit_of = (s["h"].abs().amax(1, keepdim=True) / 64)
    near(s["h"], act * up, unit_of * 1.01 + 1e-30)
    near(unit.grads[2], mm(dy.t(), s["h"]),
         mm(dy.abs().t(), s["h"].abs()) * n * 2 * F32 + mm(dy_tol.t(), s["h"].abs()))
    both = torch.cat((dh * up * slope, dh * act), 1)
    factor = torch.cat(((up * slope).abs(), act.abs()), 1)
    both_tol = torch.cat((dh_tol, dh_tol), 1) * factor
    # the function's own error: below 2^-18 of its terms at these arguments (|gate| < 40)
    both_tol = both_tol + torch.cat((dh, dh), 1).abs() * torch.cat((up.abs() * (sig + gate.abs() * sig), act.abs()), 1) * 2.0 ** -18
    both_tol = both_tol + (both.abs() + both_tol) * BF
    assert float(gate.abs().max()) < 40
    near(unit.both, both, both_tol)
    near(unit.grads[1], mm(both.t(), s["x"]),
         mm(both.abs().t(), s["x"].abs()) * n * 2 * F32 + mm(both_tol.t(), s["x"].abs()))
    back, back_tol = product(both, w[1], both_tol)
    dx = dy + back
    dx_tol = dy_tol + back_tol + (dx.abs() + dy_tol + back_tol) * BF
    near(unit.dx, dx, dx_tol)
    rows = torch.zeros_like(w[0])
    scale = math.sqrt(ex.DIM)
    want = rows.clone().index_add_(0, tokens, unit.dx.double()) * scale
    tol = rows.clone().index_add_(0, tokens, unit.dx.double().abs()) * scale * (n + 2) * F32
    near(unit.grads[0], want, tol)
    # padding behind the parameters keeps what the caller had there
    total = unit.layout["total"]
    assert bool((unit.grad[total:] == 7).all())


def test_the_step_from_them_is_the_oracles(ex, orc):
    """Two whole rounds; each step's master, slot and payload are the oracle's bits."""
    n = 200
    unit = ex.Unit(n)
    size = unit.layout["shard"]
    p, m, v = to_host(unit.opt.master).copy(), np.zeros(size, np.float32), np.zeros(size, np.float32)
    sc = orc.make_scaler(2.0 ** 10, True)
    for k in range(2):
        tokens, targets = batch_of(ex, n, 10 + k)
        unit.gather()
        _, d = ex.loss_and_gradient(unit.forward(tokens), targets, unit.opt.state.field("loss_scale"))
        unit.backward(tokens, d)
        grad = to_host(unit.grad).copy()
        unit.step()
        res = orc.shard_step(grad=grad, grad_dtype=orc.F32, master=p, exp_avg=m, exp_avg_sq=v, scaler=sc,
                             hp=orc.Hparams(**ex.HP), param_dtype=orc.BF16, quant_block=256)
        assert_bitwise(to_host(unit.opt.master), p, "master at step %d" % k)
        assert_bitwise(to_host(unit.flat), res["lp"], "slot at step %d" % k)
        q, scales = orc.quant_int8(res["lp"], orc.BF16, 256)
        assert np.array_equal(unit.codes.cpu().numpy(), q)
        assert_bitwise(unit.scales.cpu().numpy(), scales, "scales at step %d" % k)


def test_an_overflow_in_the_activations_skips_the_step(ex):
    unit = ex.Unit(64)
    tokens, targets = batch_of(ex, 64, 5)
    before = unit.opt.master.clone()
    unit.gather()
    _, d = ex.loss_and_gradient(unit.forward(tokens), targets, 1024.0)
    unit.saved["gate"].exponents[3, 2] = 255                  # as an infinity there would have left it
    unit.backward(tokens, d)
    unit.step()
    st = unit.opt.state.read()
    assert st.last_skipped == 1 and st.loss_scale == 512.0
    assert torch.equal(unit.opt.master, before)


def test_a_captured_round_replays_as_an_eager_one(ex):
    n = 256
    eager, graphed = ex.Unit(n), ex.Unit(n)
    tokens, targets = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda")

    def round_of(unit):
        unit.gather()
        loss, d = ex.loss_and_gradient(unit.forward(tokens), targets, unit.opt.state.field("loss_scale"))
        unit.backward(tokens, d)
        unit.step()
        return loss

    round_of(ex.Unit(n))                                      # warm: kernels and libraries loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss_g = round_of(graphed)
    graphed2 = ex.Unit(n)                                     # capture itself ran nothing
    assert torch.equal(graphed.opt.master, graphed2.opt.master)
    for k in range(3):
        a, b = batch_of(ex, n, 20 + k)
        tokens.copy_(a)
        targets.copy_(b)
        loss = round_of(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, loss_g)
        assert torch.equal(eager.grad, graphed.grad) and torch.equal(eager.opt.master, graphed.opt.master)
        assert torch.equal(eager.codes, graphed.codes)


def test_the_example_runs(ex):
    losses, unit = ex.train(steps=12, batch=8, length=16)
    assert len(losses) == 12 and all(math.isfinite(v) for v in losses)
    st = unit.opt.state.read()
    assert st.step + (st.last_skipped > 0) >= 1 and math.isfinite(st.last_norm)
