"""The step over a list of tensors on the GPU against the definition in 64 bits:
statistics per tensor, the update with 32-bit and 8-bit states, sizes around
rows, tiles and spans, gradients and copies at any offset, skipped steps,
streams, capture, and memory around the tensors."""
import math
import random

import numpy as np
import pytest
import torch

from harness import assert_bitwise, to_host
from list_reference import ROW, ListReference, hold_in_fp32

pytestmark = pytest.mark.gpu

HP = dict(lr=3e-4, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.01, max_grad_norm=0.5)
SIZES = {
    "one": [1],
    "rows": [255, 256, 257, 1, 511, 513],
    "tiles": [1023, 1024, 1025, 2047, 2048, 2049, 0, 3, 4097, 8191, 8193, 1793],
    "spans": [4095, 4096, 4097, 12289, 70001, 2],
    "many": [1 + (37 * k) % 700 for k in range(400)],
    "large": [3_000_017, 5, 1_200_256],
}


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    assert torch.cuda.is_available()
    return m


def lay_out(tensors, layout, dtype):
    """Device tensors of the values: "packed" back to back from the second
    element of a buffer on (any offset), "own" one allocation each."""
    if layout == "own":
        return None, [torch.tensor(t, dtype=dtype, device="cuda") for t in tensors]
    buf = torch.full((sum(len(t) for t in tensors) + 9,), 7.0, dtype=dtype, device="cuda")
    out, at = [], 1
    for t in tensors:
        out.append(buf[at:at + len(t)])
        out[-1].copy_(torch.tensor(t, dtype=dtype))
        at += len(t)
    return buf, out


def values(n, seed, sigma):
    g = np.random.default_rng(seed)
    return [g.standard_normal(x) * sigma * 10.0 ** g.uniform(-1, 1) for x in n]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["own", "packed"])
@pytest.mark.parametrize("sizes", sorted(SIZES))
def test_statistics(zf, sizes, layout, dtype):
    n = SIZES[sizes]
    _, grads = lay_out(values(n, 3, 0.1), layout, dtype)
    plan = zf.MultiPlan(n, dtype)
    plan.bind(grads)
    st = zf.StepState(1024.0, True)
    want = [float((g.double().cpu() / 1024.0).square().sum()) for g in grads]
    # two fp64 sums of x terms >= 0 in different orders
    def near(got, ref, terms):
        assert abs(got - ref) <= max(1e-12, terms * 2.0 ** -53) * ref, (got, ref)
    for call in range(3):
        zf.zero_multi_unscale_norm(plan, st, reset=True)
        got = plan.tensor_sumsq.cpu().numpy()
        for k, x in enumerate(n):
            near(got[k], want[k], x)
        near(st.read().sumsq, sum(want), sum(n))
        assert st.read().overflow == 0
        if call == 0:
            first = got.copy()
        assert np.array_equal(first, got)                  # one order, every time
    zf.zero_multi_unscale_norm(plan, st)                   # added to what is there
    near(st.read().sumsq, 2 * sum(want), 2 * sum(n))
    for k, bad in ((len(n) - 1, float("inf")), (0, float("nan"))):
        if n[k] == 0:
            continue
        keep = grads[k][-1].clone()
        grads[k][-1] = bad
        zf.zero_multi_unscale_norm(plan, st, reset=True)
        assert st.read().overflow == 1
        s = plan.tensor_sumsq.cpu()
        assert not math.isfinite(s[k]) and (len(n) == 1 or math.isfinite(s[k - 1]))
        grads[k][-1] = keep
        zf.zero_multi_unscale_norm(plan, st)
        assert st.read().overflow == 1                     # an OR without reset
    zf.zero_multi_unscale_norm(plan, st, reset=True)
    assert st.read().overflow == 0


def make(zf, n, bits, dtype, param, layout, scale=1024.0, hp=HP, seed=11, **kw):
    r = random.Random(len(n))
    lr = [r.choice((1.0, 0.1, 0.0, 2.5)) for _ in n]
    wd = [r.choice((1.0, 0.0, 3.0)) for _ in n]
    masters = [torch.tensor(t, dtype=torch.float32, device="cuda") for t in values(n, 5, 0.02)]
    opt = zf.TensorListOptimizer(masters, hp, state_bits=bits, loss_scale=scale, lr_mult=lr,
                                 decay_mult=wd, seed=seed, grad_dtype=dtype, param_dtype=param, **kw)
    ref = ListReference(n, hp, lr_mult=lr, decay_mult=wd, seed=seed)
    copies = (None, None)
    if param is not None:
        copies = lay_out([np.zeros(x) for x in n], layout, param)
    return opt, ref, copies


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def snapshot(opt):
    out = [f64(opt.master), f64(opt.exp_avg), f64(opt.exp_avg_sq)]
    if opt.exp_avg_scale is not None:
        out += [opt.exp_avg_scale.cpu().numpy(), opt.exp_avg_sq_scale.cpu().numpy()]
    return out


def check_step(opt, ref, grads, before, t, scale, copies, bits):
    g = [f64(x) for x in grads]
    want = ref.step(g, *before[:3], t, scale, bits, *before[3:])
    after = snapshot(opt)
    off = np.abs(after[0] - want["p"]) - want["p_err"]
    assert off.max(initial=-1) <= 0, ("master", int(off.argmax()), off.max())
    if bits == 32:
        for key, x in (("m", after[1]), ("v", after[2])):
            off = np.abs(x - want[key]) - want[key + "_err"]
            assert off.max(initial=-1) <= 0, (key, int(off.argmax()), off.max())
    else:
        ref.check_codes(want, t, after[1], after[2], after[3], after[4])
    if copies is not None:
        for k, (c, mst) in enumerate(zip(copies, opt.views(opt.master))):
            assert torch.equal(c, mst.to(c.dtype)), ("copy", k)
    st = opt.state.read()
    assert abs(st.last_norm - want["norm"]) <= 1e-10 * want["norm"]
    assert st.step == t and st.last_skipped == 0
    # the padding of every tensor's last row
    for k, x in enumerate(ref.n):
        a, b = int(ref.row0[k]) * ROW + x, int(ref.row0[k + 1]) * ROW
        assert not any(s[a:b].any() for s in after[:3]), ("padding", k)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,param", [(torch.bfloat16, torch.bfloat16),
                                         (torch.float16, torch.float16),
                                         (torch.float32, torch.bfloat16), (torch.float32, None),
                                         (torch.float16, None), (torch.bfloat16, torch.float16)])
@pytest.mark.parametrize("layout", ["own", "packed"])
@pytest.mark.parametrize("sizes", sorted(SIZES))
def test_steps(zf, sizes, layout, dtype, param, bits):
    """Three steps, each from the library's own state; the first from zeros."""
    n = SIZES[sizes]
    scale = 1024.0
    opt, ref, (buf, copies) = make(zf, n, bits, dtype, param, layout, scale)
    grads = None
    for t in (1, 2, 3):
        vals = values(n, 100 + t, 0.3)
        vals[0][: len(vals[0]) // 2] = 0.0                 # rows no gradient reaches
        gbuf, grads = lay_out([v * 1.0 for v in vals], layout, dtype)
        opt.bind(grads, copies)
        before = snapshot(opt)
        opt.step()
        torch.cuda.synchronize()
        check_step(opt, ref, grads, before, t, scale, copies, bits)
        if buf is not None:                                # nothing around the copies
            assert float(buf[0]) == 7.0 and torch.all(buf[1 + sum(n):] == 7.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("sizes", ["spans", "large"])
def test_states_in_8_bits_are_fp32_operations_one_by_one(zf, sizes, dtype):
    """Every code and scale of five steps, bit for bit: a rounding that fell the
    other way would be a whole code off."""
    n = SIZES[sizes]
    opt, ref, _ = make(zf, n, 8, dtype, None, "own", 256.0)
    for t in range(1, 6):
        _, grads = lay_out(values(n, 60 + t, 0.3), "packed", dtype)
        opt.bind(grads)
        before = snapshot(opt)
        opt.step()
        coef = opt.state.read().last_coef
        want = hold_in_fp32(ref.arena([f64(x) for x in grads]), *before[1:], HP,
                            np.float32(1 / 256) * np.float32(coef), t, 11)
        for name, a, b in zip(("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"),
                              snapshot(opt)[1:], want):
            assert np.array_equal(a, b), (t, name, int(np.sum(a != b)))


@pytest.mark.parametrize("bits", [32, 8])
def test_gaps_between_packed_tensors_stay(zf, bits):
    """Every second tensor of a buffer is in the list: the others keep their
    values, whatever words they share with the list's."""
    n = [1 + (311 * k) % 5000 for k in range(60)]
    at = np.concatenate(([0], np.cumsum(n)))
    grad = torch.randn(int(at[-1]), device="cuda").to(torch.bfloat16)
    copy = torch.full((int(at[-1]),), 3.0, dtype=torch.bfloat16, device="cuda")
    own = [slice(int(at[k]), int(at[k + 1])) for k in range(1, 60, 2)]
    masters = [torch.randn(s.stop - s.start, device="cuda") for s in own]
    opt = zf.TensorListOptimizer(masters, HP, state_bits=bits)
    opt.bind([grad[s] for s in own], [copy[s] for s in own])
    opt.step()
    mine = torch.zeros_like(copy, dtype=torch.bool)
    for s, m in zip(own, opt.views(opt.master)):
        assert torch.equal(copy[s], m.to(torch.bfloat16))
        mine[s] = True
    assert torch.all(copy[~mine] == 3.0)


@pytest.mark.parametrize("n", [5, 1024, 300_001, 40_000_003])
def test_one_tensor_equals_the_flat_step(zf, n):
    """32-bit states and factors of one: the flat shard's step, bit for bit."""
    torch.manual_seed(n)
    master = torch.randn(n, device="cuda") * 0.02
    hp = dict(HP, max_grad_norm=0.0)                       # the norms' orders differ
    flat = zf.ShardOptimizer(master.clone(), hp, loss_scale=65536.0, dynamic=True, window=2)
    lst = zf.TensorListOptimizer([master], hp, loss_scale=65536.0, dynamic=True, window=2,
                                 grad_dtype=torch.float16, param_dtype=torch.float16)
    slot = torch.zeros(n, dtype=torch.float16, device="cuda")
    copy = torch.zeros(n, dtype=torch.float16, device="cuda")
    for step in range(4):
        g = (torch.randn(n, device="cuda") * 30).half()
        if step == 2:
            g[n // 2] = float("inf")
        flat.step_from_reduced(g, slot, 0)
        lst.bind([g], [copy])
        lst.step()
        for a, b, name in ((flat.master, lst.master[:n], "master"),
                           (flat.exp_avg, lst.exp_avg[:n], "exp_avg"),
                           (flat.exp_avg_sq, lst.exp_avg_sq[:n], "exp_avg_sq"),
                           (slot, copy, "copy")):
            assert_bitwise(to_host(a), to_host(b), "%s after step %d" % (name, step))
        a, b = flat.state.read(), lst.state.read()
        for f in ("step", "good_steps", "loss_scale", "last_skipped", "beta1_pow", "beta2_pow",
                  "last_coef", "sumsq", "overflow"):
            assert getattr(a, f) == getattr(b, f), f


@pytest.mark.parametrize("bits", [32, 8])
def test_a_skipped_step_writes_nothing(zf, bits):
    n = SIZES["tiles"]
    opt, ref, (buf, copies) = make(zf, n, bits, torch.float16, torch.float16, "packed", 256.0,
                                   dynamic=True)
    _, grads = lay_out(values(n, 1, 0.3), "packed", torch.float16)
    opt.bind(grads, copies)
    opt.step()
    arenas = [opt.master, opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8), buf]
    if bits == 8:
        arenas += [opt.exp_avg_scale, opt.exp_avg_sq_scale]
    before = [x.clone() for x in arenas]
    grads[4][7] = float("nan")
    opt.step()
    st = opt.state.read()
    assert (st.last_skipped, st.step, st.loss_scale, st.good_steps) == (1, 1, 128.0, 0)
    assert all(torch.equal(a, b) for a, b in zip(arenas, before))
    grads[4][7] = 1.0
    snap = snapshot(opt)
    opt.step()
    check_step(opt, ref, grads, snap, 2, 128.0, copies, bits)
    # another rank's overflow skips too
    opt.state.set_remote(0.0, 1)
    before = [x.clone() for x in arenas]
    opt.step()
    assert opt.state.read().last_skipped == 1
    assert all(torch.equal(a, b) for a, b in zip(arenas, before))


@pytest.mark.parametrize("bits", [32, 8])
def test_without_statistics(zf, bits):
    """No norm, no clip, no test for overflow: the update alone."""
    n = SIZES["tiles"]
    hp = dict(HP, max_grad_norm=0.0)
    with pytest.raises(ValueError, match="statistics"):
        make(zf, n, bits, torch.bfloat16, None, "own", statistics=False)
    opt, ref, _ = make(zf, n, bits, torch.bfloat16, None, "own", 1.0, hp=hp, statistics=False)
    _, grads = lay_out(values(n, 8, 0.3), "packed", torch.bfloat16)
    opt.bind(grads)
    before = snapshot(opt)
    opt.step()
    want = ref.step([f64(x) for x in grads], *before[:3], 1, 1.0, bits, *before[3:])
    assert np.all(np.abs(snapshot(opt)[0] - want["p"]) <= want["p_err"])
    st = opt.state.read()
    assert (st.last_norm, st.step, st.last_coef) == (0.0, 1, 1.0)
    # a gradient that is not finite reaches its own row only
    a = int(ref.row0[9]) * ROW + 5
    grads[9][5] = float("nan")
    opt.step()
    got = snapshot(opt)
    assert np.isnan(got[0][a]) and np.isnan(got[1][a])
    assert np.sum(~np.isfinite(got[0])) == 1 and np.sum(~np.isfinite(got[1])) == 1
    if bits == 8:
        assert np.all(np.isfinite(got[3])) and np.all(np.isfinite(got[4]))
        row = int(ref.row0[9])
        assert got[3][row] > 0 and got[2][a] == 0


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [0.0, 1e-30, 3e38])
def test_extreme_gradients(zf, bits, value):
    """Zeros keep every state at zero; tiny squares underflow to a second moment
    of zero (the update is then m/eps); huge ones meet the largest scale."""
    n = [256, 700]
    hp = dict(HP, max_grad_norm=0.0, lr=1e-3)
    opt = zf.TensorListOptimizer([torch.ones(x, device="cuda") for x in n], hp, state_bits=bits,
                                 loss_scale=1.0, grad_dtype=torch.float32, param_dtype=None)
    opt.bind([torch.full((x,), value, device="cuda") for x in n])
    opt.step()
    p = opt.views(opt.master)[1]
    if value == 0.0:
        assert torch.all(p == p[0]) and abs(float(p[0]) - (1 - 1e-5)) < 1e-7
        assert not opt.exp_avg.float().any() and not opt.exp_avg_sq.float().any()
    elif value == 1e-30:
        # m/bc1 = 1e-30, v = 0 in fp32: p moves by lr * 1e-30 / 1e-8
        assert not opt.views(opt.exp_avg_sq)[1].float().any()
        assert abs(float(p[0]) - (1 - 1e-5)) < 1e-7
    else:
        # v overflows to infinity: the update vanishes, the state stays a number
        assert abs(float(p[0]) - (1 - 1e-5)) < 1e-7
        if bits == 8:
            assert torch.all(torch.isfinite(opt.views(opt.exp_avg_sq)[1].float()))


def rounding_corners():
    """fp32 patterns where a 16-bit rounding decides: every binary16 value of
    the exponents' ends, the midpoints between neighbours and one fp32 step to
    either side, the borders of overflow and underflow, and what is no number."""
    h = np.arange(0x7C00, dtype=np.uint16)                 # every finite binary16 >= 0
    f = h.view(np.float16).astype(np.float32)
    mid = (f[:-1].astype(np.float64) + f[1:].astype(np.float64)) / 2
    b = (np.arange(0x0000, 0x7F80, 7, dtype=np.uint32) << 16)    # bfloat16 values and midpoints
    x = np.concatenate((f, mid.astype(np.float32), b.view(np.float32),
                        (b + 0x8000).view(np.float32),
                        np.array([65519.996, 65520.0, 65504.0, 2.0 ** -25, 2.0 ** -24, 2.0 ** -26,
                                  1e-45, 3.4e38, 0.0, np.inf], np.float32)))
    bits = np.concatenate([x.view(np.uint32) + d for d in (0, 1)] + [x.view(np.uint32)[1:] - 1])
    bits = bits[bits <= 0x7F800000]
    bits = np.concatenate((bits, bits | 0x80000000,
                           np.array([0x7FC00000, 0xFFC00000, 0x7F800001], np.uint32)))
    return bits.astype(np.uint32).view(np.float32)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1])
def test_copies_round_to_nearest(zf, bits, param, shift):
    """No rate and no decay: the master stays, and its copy is the nearest
    16-bit value, ties to even (numpy's and torch's casts on the host)."""
    x = rounding_corners()
    hp = dict(HP, lr=0.0, weight_decay=0.0, max_grad_norm=0.0)
    opt = zf.TensorListOptimizer([torch.from_numpy(x).cuda()], hp, state_bits=bits, statistics=False,
                                 loss_scale=1.0, grad_dtype=torch.float32, param_dtype=param)
    buf = torch.zeros(len(x) + 4, dtype=param, device="cuda")
    opt.bind([torch.zeros(len(x), device="cuda")], [buf[shift:shift + len(x)]])
    opt.step()
    assert_bitwise(to_host(opt.master[:len(x)])[~np.isnan(x)], x[~np.isnan(x)], "master")
    got = to_host(buf[shift:shift + len(x)])
    if param == torch.float16:
        with np.errstate(over="ignore"):
            want = x.astype(np.float16).view(np.uint16)
        quiet = 0x7E00
    else:
        want = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
        quiet = 0x7FC0
    nan = np.isnan(x)
    assert np.all(got[nan] & 0x7FFF == quiet)
    assert_bitwise(got[~nan], want[~nan], "copy")


def test_first_moment_ties_go_to_even(zf):
    """beta1 = 0 and a row whose largest gradient is 448: the scale is one, and
    every value halfway between two e4m3 codes is held as the even one."""
    assert np.float32(448) * np.float32(1 / 448) == 1
    code = np.arange(1, 0x7E, dtype=np.uint8)
    vals = torch.from_numpy(code).view(torch.float8_e4m3fn).float().numpy()   # up to 416
    mid = ((vals[:-1].astype(np.float64) + vals[1:]) / 2).astype(np.float32)
    g = np.zeros(512, np.float32)
    g[0] = g[256] = 448.0
    g[1:1 + len(mid)] = mid
    g[257:257 + len(mid)] = -mid
    hp = dict(HP, beta1=0.0, max_grad_norm=0.0)
    opt = zf.TensorListOptimizer([torch.zeros(512, device="cuda")], hp, state_bits=8, loss_scale=1.0,
                                 grad_dtype=torch.float32, param_dtype=None)
    opt.bind([torch.from_numpy(g).cuda()])
    opt.step()
    assert opt.exp_avg_scale.tolist() == [1.0, 1.0]
    from list_reference import nearest_e4m3
    assert np.array_equal(f64(opt.exp_avg), nearest_e4m3(g.astype(np.float64)))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_past_two_to_the_31(zf, bits):
    """Elements, bytes and rows past 32 bits: the ends and the border of one
    long tensor behind another, against the same elements on their own."""
    n = [700, (1 << 31) + 1027]
    hp = dict(HP, max_grad_norm=0.0)
    def packed(dtype):
        t = torch.zeros(n[0] + n[1] + 1, dtype=dtype, device="cuda")
        return t, [t[1:1 + n[0]], t[1 + n[0]:]]
    gbuf, grads = packed(torch.bfloat16)
    cbuf, copies = packed(torch.bfloat16)
    cuts = [slice(0, 2048), slice((1 << 31) - 2048, (1 << 31) + 512), slice(n[1] - 1027, n[1])]
    torch.manual_seed(3)
    for c in cuts:
        grads[1][c] = torch.randn(c.stop - c.start, device="cuda").to(torch.bfloat16)
    grads[0].normal_()
    masters = [torch.zeros(x, device="cuda") for x in n]
    opt = zf.TensorListOptimizer(masters, hp, state_bits=bits, loss_scale=1.0)
    del masters
    opt.bind(grads, copies)
    opt.step()
    want = sum(float(grads[1][c].double().square().sum()) for c in (cuts[0], cuts[1], cuts[2])) - \
        float(grads[1][slice(max(cuts[1].start, cuts[2].start), cuts[1].stop)].double().square().sum())
    got = opt.plan.tensor_sumsq.tolist()
    assert abs(got[1] - want) <= 1e-9 * want
    first = float(grads[0].double().square().sum())
    assert abs(got[0] - first) <= 1e-9 * first
    p = opt.views(opt.master)[1]
    for c in cuts:
        ref = ListReference([c.stop - c.start], hp)
        z = np.zeros(ref.row0[-1] * ROW)
        sc = (np.zeros(ref.row0[-1], np.float32),) * 2 if bits == 8 else ()
        w = ref.step([f64(grads[1][c])], z, z, z, 1, 1.0, bits, *sc)
        k = c.stop - c.start
        assert np.all(np.abs(f64(p[c]) - w["p"][:k]) <= w["p_err"][:k])
        assert torch.equal(copies[1][c], p[c].to(torch.bfloat16))
    assert not p[4096:1 << 20].any() and float(cbuf[0]) == 0.0


def test_second_moment_rounding_is_unbiased(zf):
    """From one state the rounded second moments of many seeds have its mean:
    256 * 64 elements and 32 seeds; a code's step is at most a quarter of its
    value, so the mean of N rounded values is within 6 * 0.25/2 / sqrt(N)."""
    n = [256 * 64]
    hp = dict(HP, max_grad_norm=0.0, beta2=0.9)
    torch.manual_seed(1)
    g = torch.rand(n[0], device="cuda") + 0.5
    ratios = []
    for seed in range(32):
        opt = zf.TensorListOptimizer([torch.zeros(n[0], device="cuda")], hp, state_bits=8,
                                     loss_scale=1.0, grad_dtype=torch.float32, param_dtype=None,
                                     seed=seed)
        opt.bind([g])
        opt.step()
        v = opt.exp_avg_sq.double() * opt.exp_avg_sq_scale.double().repeat_interleave(256)
        ratios.append((v / (0.1 * g.double() ** 2)).mean())
    mean = float(torch.stack(ratios).mean())
    assert abs(mean - 1) <= 6 * 0.125 / math.sqrt(32 * n[0]), mean


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", ["tiles", "large"])
def test_captured_step_replays_equal_eager_steps(zf, bits, sizes):
    n = SIZES[sizes]
    pair = [make(zf, n, bits, torch.float16, torch.float16, "packed", 256.0, dynamic=True,
                 window=2) for _ in range(2)]
    _, grads = lay_out(values(n, 2, 0.3), "packed", torch.float16)
    for opt, _, (_, copies) in pair:
        opt.bind(grads, copies)
    (eager, _, (buf_e, _)), (graphed, _, (buf_g, _)) = pair
    eager.step()
    graphed.step()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            graphed.step()
            with pytest.raises(RuntimeError, match="capture"):
                graphed.bind(grads, pair[1][2][1])
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert graphed.state.read().step == 1
    for step in range(5):
        vals = values(n, 50 + step, 0.3)
        for g, v in zip(grads, vals):
            g.copy_(torch.tensor(v, dtype=torch.float16))
        if step == 2:
            grads[0][0] = float("inf")
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert bytes(eager.state.read())[:88] == bytes(graphed.state.read())[:88]
        for a, b in zip(snapshot(eager), snapshot(graphed)):
            assert np.array_equal(a, b)
        assert torch.equal(buf_e, buf_g)
    assert eager.state.read().step == 5


def test_on_another_stream(zf):
    """A step on a stream of its own, ordered by the caller."""
    n = SIZES["spans"]
    a, _, (_, ca) = make(zf, n, 8, torch.bfloat16, torch.bfloat16, "own")
    b, _, (_, cb) = make(zf, n, 8, torch.bfloat16, torch.bfloat16, "own")
    _, grads = lay_out(values(n, 2, 0.3), "own", torch.bfloat16)
    a.bind(grads, ca)
    b.bind(grads, cb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        a.step()
        b.step(stream=s)
    torch.cuda.synchronize()
    for x, y in zip(snapshot(a), snapshot(b)):
        assert np.array_equal(x, y)


def test_lists_and_shards_share_one_step(zf):
    """Statistics of two lists into one state, one clip over both."""
    n = [[3000, 5], [700, 12_345]]
    st = zf.StepState(1.0, False)
    hp = zf.zero_adamw_hparams_t(**HP)
    plans, arenas, all_g = [], [], []
    for k, m in enumerate(n):
        _, g = lay_out(values(m, 20 + k, 1.0), "own", torch.float32)
        plan = zf.MultiPlan(m, torch.float32, None, 32)
        plan.bind(g)
        plans.append(plan)
        all_g += g
        arenas.append([torch.zeros(plan.rows * ROW, device="cuda") for _ in range(3)])
        zf.zero_multi_unscale_norm(plan, st)
    for k, (plan, (p, m, v)) in enumerate(zip(plans, arenas)):
        zf.zero_multi_adamw_step(plan, p, m, v, hp, st, finalize=k == 1)
    got = st.read()
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in all_g))
    assert abs(got.last_norm - norm) <= 1e-10 * norm and got.step == 1
    assert abs(got.last_coef - HP["max_grad_norm"] / norm) <= 1e-6 * got.last_coef
    # m after one step from zero: (1 - beta1) * clipped gradient
    m = arenas[1][1][3 * ROW:3 * ROW + 12_345].double()
    want = all_g[3].double() * (got.last_coef * (1 - HP["beta1"]))
    assert float((m - want).abs().max()) <= 4 * 2.0 ** -24 * float(want.abs().max())


def test_an_empty_list_still_advances_the_state(zf):
    opt = zf.TensorListOptimizer([torch.zeros(0, device="cuda")], HP, state_bits=8, loss_scale=4.0)
    opt.bind([torch.zeros(0, dtype=torch.bfloat16, device="cuda")],
             [torch.zeros(0, dtype=torch.bfloat16, device="cuda")])
    opt.step()
    st = opt.state.read()
    assert (st.step, st.last_norm, st.last_skipped) == (1, 0.0, 0)
    assert opt.plan.tensor_sumsq.tolist() == [0.0]
    plan = zf.MultiPlan([], torch.float32)
    plan.bind([])
    state = zf.StepState(1.0, False)
    state.field("sumsq").fill_(3.0)
    zf.zero_multi_unscale_norm(plan, state)
    assert state.read().sumsq == 3.0
    zf.zero_multi_unscale_norm(plan, state, reset=True)
    assert (state.read().sumsq, state.read().overflow) == (0.0, 0)


def test_bind_refusals(zf):
    opt = zf.TensorListOptimizer([torch.zeros(8, device="cuda")], HP)
    g = torch.zeros(8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(RuntimeError, match="bind"):
        opt.step()
    with pytest.raises(ValueError, match="params"):
        opt.bind([g])
    with pytest.raises(ValueError, match="bfloat16"):
        opt.bind([g.half()], [g])
    with pytest.raises(ValueError, match="elements"):
        opt.bind([g[:7]], [g])
    with pytest.raises(ValueError, match="contiguous"):
        opt.bind([torch.zeros(16, dtype=torch.bfloat16, device="cuda")[::2]], [g])
    with pytest.raises(ValueError, match="lr_mult"):
        opt.plan.bind([g], [g.clone()], lr_mult=[1.0, 2.0])
    with pytest.raises(zf.ZeroError):
        opt.plan.bind([g], [g.clone()], lr_mult=[-1.0])
    opt.bind([g], [g.clone()])
    opt.step()


def test_example_trains(zf):
    """The example's MLP learns with 8-bit states as with 32-bit ones."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import list_adamw
    final = {}
    for bits in (32, 8):
        losses, opt = list_adamw.train(bits, 150)
        assert opt.state.read().step == 150
        assert losses[-1] < 0.2 * losses[0], (bits, losses[0], losses[-1])
        final[bits] = losses[-1]
    assert final[8] < 2 * final[32] + 0.01, final
