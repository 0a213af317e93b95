"""The step over long lists (more than 2048 spans) on the GPU, which take tiles
of four rows, the fold as a launch of its own and launches over slices of the
tiles: the definition in 64 bits, the 8-bit states bit for bit, skipped steps,
steps without statistics, capture, and slices."""
import numpy as np
import pytest
import torch

import list_reference
from list_reference import ROW, ListReference, hold_in_fp32, mix
from test_gpu_multi_list import HP, check_step, f64, lay_out, make, snapshot, values

pytestmark = pytest.mark.gpu

SIZES = {
    # a span per tensor, with tiles that are whole and tiles of 1 to 4 rows
    "tensors": [1 + (1237 * k) % 2999 for k in range(2100)],
    # a row per tensor: no whole tile
    "rows": [1 + (53 * k) % 250 for k in range(2300)] + [0],
    # few tensors, long by their elements
    "elements": [9_000_001, 1793, 2050, 5003, 4097, 3, 0, 255],
}
SLICED = 131072 * 1024 + 70_001      # more tiles than one launch takes


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    assert torch.cuda.is_available()
    return m


def check_arenas(ref, grads, before, after, t, scale, bits):
    want = ref.step([f64(x) for x in grads], *before[:3], t, scale, bits, *before[3:])
    assert np.all(np.abs(after[0] - want["p"]) <= want["p_err"])
    if bits == 32:
        assert np.all(np.abs(after[1] - want["m"]) <= want["m_err"])
        assert np.all(np.abs(after[2] - want["v"]) <= want["v_err"])
    else:
        ref.check_codes(want, t, *after[1:])


PAIRS = [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
         (torch.float32, torch.bfloat16), (torch.float32, None), (torch.float16, None),
         (torch.bfloat16, torch.float16)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes,layout,dtype,param", [("tensors", "packed") + p for p in PAIRS] +
                         [("tensors", "own") + PAIRS[1]] + [("rows", "packed") + p for p in PAIRS[:4]] +
                         [("elements", "packed") + p for p in PAIRS[:2]])
def test_steps(zf, sizes, layout, dtype, param, bits):
    """Two steps, each from the library's own state; the first from zeros."""
    n = SIZES[sizes]
    opt, ref, (buf, copies) = make(zf, n, bits, dtype, param, layout)
    assert opt.plan._plan.tile_rows == 4
    for t in (1, 2):
        vals = values(n, 100 + t, 0.3)
        vals[0][: len(vals[0]) // 2] = 0.0                 # rows no gradient reaches
        _, grads = lay_out(vals, layout, dtype)
        opt.bind(grads, copies)
        before = snapshot(opt)
        opt.step()
        check_step(opt, ref, grads, before, t, 1024.0, copies, bits)
        if buf is not None:                                # nothing around the copies
            assert float(buf[0]) == 7.0 and torch.all(buf[1 + sum(n):] == 7.0)


@pytest.mark.parametrize("sizes,dtype", [("tensors", torch.bfloat16), ("tensors", torch.float16),
                                         ("tensors", torch.float32), ("rows", torch.bfloat16),
                                         ("elements", torch.float16)])
def test_states_in_8_bits_are_fp32_operations_one_by_one(zf, sizes, dtype):
    """Every code and scale of three steps, bit for bit."""
    n = SIZES[sizes]
    opt, ref, _ = make(zf, n, 8, dtype, None, "own", 256.0)
    for t in (1, 2, 3):
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
def test_a_skipped_step_writes_nothing(zf, bits):
    n = SIZES["tensors"]
    opt, ref, (buf, copies) = make(zf, n, bits, torch.float16, torch.float16, "packed", 256.0,
                                   dynamic=True)
    _, grads = lay_out(values(n, 1, 0.3), "packed", torch.float16)
    opt.bind(grads, copies)
    opt.step()
    arenas = [opt.master, opt.exp_avg.view(torch.uint8), opt.exp_avg_sq.view(torch.uint8), buf]
    if bits == 8:
        arenas += [opt.exp_avg_scale, opt.exp_avg_sq_scale]
    before = [x.clone() for x in arenas]
    grads[-1][0] = float("inf")
    opt.step()
    st = opt.state.read()
    assert (st.last_skipped, st.step, st.loss_scale, st.good_steps) == (1, 1, 128.0, 0)
    assert all(torch.equal(a, b) for a, b in zip(arenas, before))
    grads[-1][0] = 1.0
    snap = snapshot(opt)
    opt.step()
    check_step(opt, ref, grads, snap, 2, 128.0, copies, bits)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", ["tensors", "elements"])
def test_without_statistics(zf, sizes, bits):
    """The step's scalars in a launch of their own, then the update alone."""
    n = SIZES[sizes]
    hp = dict(HP, max_grad_norm=0.0)
    opt, ref, (_, copies) = make(zf, n, bits, torch.bfloat16, torch.bfloat16, "packed", 1.0, hp=hp,
                                 statistics=False)
    _, grads = lay_out(values(n, 8, 0.3), "packed", torch.bfloat16)
    opt.bind(grads, copies)
    before = snapshot(opt)
    opt.step()
    check_arenas(ref, grads, before, snapshot(opt), 1, 1.0, bits)
    st = opt.state.read()
    assert (st.last_norm, st.step, st.last_coef) == (0.0, 1, 1.0)
    for c, p in zip(copies, opt.views(opt.master)):
        assert torch.equal(c, p.to(c.dtype))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step_replays_equal_eager_steps(zf, bits):
    n = SIZES["tensors"]
    pair = [make(zf, n, bits, torch.float16, torch.float16, "packed", 256.0, dynamic=True,
                 window=2) for _ in range(2)]
    gbuf, grads = lay_out(values(n, 2, 0.3), "packed", torch.float16)
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
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for step in range(4):
        gbuf[1:1 + sum(n)] = torch.tensor(np.concatenate(values(n, 50 + step, 0.3)),
                                          dtype=torch.float16)
        if step == 2:
            grads[0][0] = float("inf")
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert bytes(eager.state.read())[:88] == bytes(graphed.state.read())[:88]
        for a, b in zip(snapshot(eager), snapshot(graphed)):
            assert np.array_equal(a, b)
        assert torch.equal(buf_e, buf_g)
    assert eager.state.read().step == 4


def test_slices_with_32_bits_equal_the_flat_step(zf):
    torch.manual_seed(4)
    master = torch.randn(SLICED, device="cuda") * 0.02
    hp = dict(HP, max_grad_norm=0.0)                       # the norms' orders differ
    flat = zf.ShardOptimizer(master.clone(), hp, loss_scale=1024.0)
    lst = zf.TensorListOptimizer([master], hp, loss_scale=1024.0, grad_dtype=torch.bfloat16,
                                 param_dtype=torch.bfloat16)
    slot, copy = (torch.zeros(SLICED + 3, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for _ in range(2):
        g = (torch.randn(SLICED + 3, device="cuda") * 300).bfloat16()[3:]
        flat.step_from_reduced(g, slot, 3)
        lst.bind([g], [copy[3:]])
        lst.step()
    for a, b in ((flat.master, lst.master), (flat.exp_avg, lst.exp_avg),
                 (flat.exp_avg_sq, lst.exp_avg_sq)):
        assert torch.equal(a, b[:SLICED]) and not b[SLICED:].any()
    assert torch.equal(slot, copy)


def test_slices_with_8_bits(zf, monkeypatch):
    """Rows at the start, at the border of two launches and at the end, bit for
    bit, and every copy against its master."""
    torch.manual_seed(5)
    hp = dict(HP, max_grad_norm=0.0)
    opt = zf.TensorListOptimizer([torch.randn(SLICED, device="cuda") * 0.02], hp, state_bits=8, seed=9,
                                 loss_scale=256.0, grad_dtype=torch.float16, param_dtype=torch.float16)
    copy = torch.zeros(SLICED + 2, dtype=torch.float16, device="cuda")
    border, rows = 131072 * 4, opt.plan.rows
    cuts = [(0, 8), (border - 8, border + 8), (rows - 5, rows)]
    definition = list_reference.random16

    def at(row0):
        def random16(R, t, seed):
            # the definition's rows row0 .. row0 + R: its key is mix(mix(t + seed) + row)
            assert np.array_equal(definition(R, t, seed), numbers(0, R, t, seed))
            return numbers(row0, R, t, seed)
        return random16

    def numbers(row0, R, t, seed):
        base = mix(np.array([t + seed], np.uint64))
        key = mix((base + np.arange(row0, row0 + R, dtype=np.uint64)) & np.uint64(0xFFFFFFFF))
        h = mix((key[:, None] + np.arange(64, dtype=np.uint64) * np.uint64(0x9E3779B9)) &
                np.uint64(0xFFFFFFFF))
        k = (h * np.uint64(0x2C1B3C6D)) & np.uint64(0xFFFFFFFF)
        k = k ^ (k >> np.uint64(13))
        low = np.uint64(0xFFFF)
        return np.stack((h & low, h >> np.uint64(16), k & low, k >> np.uint64(16)),
                        2).reshape(R, ROW).astype(np.float64)

    def cut(a, b):
        e = slice(a * ROW, b * ROW)
        return [f64(opt.master[e]), f64(opt.exp_avg[e]), f64(opt.exp_avg_sq[e]),
                opt.exp_avg_scale[a:b].cpu().numpy(), opt.exp_avg_sq_scale[a:b].cpu().numpy()]

    for t in (1, 2):
        g = (torch.randn(SLICED + 2, device="cuda") * 80).half()[2:]
        opt.bind([g], [copy[2:]])
        before = [cut(a, b) for a, b in cuts]
        opt.step()
        for (a, b), old in zip(cuts, before):
            monkeypatch.setattr(list_reference, "random16", at(a))
            x = f64(g[a * ROW:b * ROW])
            ref = ListReference([len(x)], hp, seed=9)
            want = hold_in_fp32(ref.arena([x]), *old[1:], hp, np.float32(1 / 256), t, 9)
            new = cut(a, b)
            for p, q in zip(new[1:], want):
                assert np.array_equal(p, q), (t, a)
            w = ref.step([x], *old[:3], t, 256.0, 8, *old[3:])
            assert np.all(np.abs(new[0] - w["p"]) <= w["p_err"]), (t, a)
        assert torch.equal(copy[2:], opt.views(opt.master)[0].half())
        assert not opt.master[SLICED:].any()
