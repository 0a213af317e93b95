"""The list entry points on the host: the plan's tables, and every refusal
before anything is launched (no GPU needed)."""
import ctypes as C

import numpy as np
import pytest
import torch

HP = dict(lr=3e-5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, max_grad_norm=1.0)
P = C.c_void_p(0x1000)


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    return m


def make(zf, numels, grad=1, param=2, bits=8, image=True):
    plan = zf.zero_multi_plan_t()
    arr = (C.c_int64 * max(len(numels), 1))(*numels)
    L = zf.lib()
    rc = L.zero_multi_plan_init(arr, len(numels), grad, param, bits, C.byref(plan), None, 0)
    if rc or not image:
        return rc, plan, None
    host = np.full(plan.image_bytes + 64, 0xAB, np.uint8)
    rc = L.zero_multi_plan_init(arr, len(numels), grad, param, bits, C.byref(plan),
                                C.c_void_p(host.ctypes.data), plan.image_bytes)
    assert np.all(host[plan.image_bytes:] == 0xAB)
    return rc, plan, host


@pytest.mark.parametrize("bits", [32, 8, 0])
@pytest.mark.parametrize("numels", [[1], [0], [256, 257, 0, 255], [4096, 1, 5000, 1 << 20], [], [9_000_001, 3],
                                    [7] * 900])
def test_plan_tables(zf, numels, bits):
    rc, plan, host = make(zf, numels, bits=bits)
    assert rc == 0
    assert plan.tile_rows == (4 if plan.n_spans > 2048 else 2 if plan.rows > 2048 else 1)
    rows = [-(-n // 256) for n in numels]
    tiles = [-(-r // plan.tile_rows) if bits else 0 for r in rows]
    spans = [-(-n // plan.span) for n in numels]
    assert (plan.total, plan.rows, plan.n_tiles, plan.n_spans) == \
        (sum(numels), sum(rows), sum(tiles), sum(spans))
    table = host[plan.tiles_off:plan.tiles_off + 4 * plan.n_tiles].view(np.int32)
    assert np.array_equal(table, np.repeat(np.arange(len(numels)), tiles))
    table = host[plan.spans_off:plan.spans_off + 4 * plan.n_spans].view(np.int32)
    assert np.array_equal(table, np.repeat(np.arange(len(numels)), spans))
    assert plan.sumsq_off + 8 * len(numels) <= plan.image_bytes
    assert plan.bind_bytes == 64 * len(numels)
    assert not host[plan.sumsq_off:plan.image_bytes].any()


def test_plan_refusals(zf):
    L = zf.lib()
    assert make(zf, [-1])[0] == -1
    assert make(zf, [4], grad=5)[0] == -1
    assert make(zf, [4], param=0)[0] == -1                 # an fp32 copy
    assert make(zf, [4], bits=16)[0] == -1
    assert make(zf, [1 << 60])[0] == -3
    assert make(zf, [1 << 55, 1 << 55, 1 << 55])[0] == -3
    assert make(zf, [1 << 45], image=False)[0] == -3       # more rows than an int32
    arr = (C.c_int64 * 1)(4)
    plan = zf.zero_multi_plan_t()
    assert L.zero_multi_plan_init(arr, 1, 1, 2, 8, None, None, 0) == -1
    assert L.zero_multi_plan_init(None, 1, 1, 2, 8, C.byref(plan), None, 0) == -1
    assert L.zero_multi_plan_init(arr, -1, 1, 2, 8, C.byref(plan), None, 0) == -1
    assert L.zero_multi_plan_init(arr, (1 << 20) + 1, 1, 2, 8, C.byref(plan), None, 0) == -3
    assert L.zero_multi_plan_init(arr, 1, 1, 2, 8, C.byref(plan), None, 0) == 0
    buf = np.zeros(plan.image_bytes + 8, np.uint8)
    at = buf.ctypes.data
    assert L.zero_multi_plan_init(arr, 1, 1, 2, 8, C.byref(plan), C.c_void_p(at), 16) == -3
    assert L.zero_multi_plan_init(arr, 1, 1, 2, 8, C.byref(plan), C.c_void_p(at + 4),
                                  plan.image_bytes) == -2
    assert not buf.any()


def test_bind_refusals(zf):
    L = zf.lib()
    rc, plan, host = make(zf, [4, 0, 300])
    image = C.c_void_p(host.ctypes.data)
    before = host.copy()

    def bind(g=(0x1000, 0, 0x2002), p=(0x3000, 0, 0x4002), lr=None, wd=None, image=image):
        ga = None if g is None else (C.c_void_p * 3)(*g)
        pa = None if p is None else (C.c_void_p * 3)(*p)
        dbl = lambda x: None if x is None else (C.c_double * 3)(*x)     # noqa: E731
        return L.zero_multi_bind(C.byref(plan), ga, pa, dbl(lr), dbl(wd), image)

    assert bind(g=None) == -1 and bind(p=None) == -1
    assert bind(g=(0x1000, 0, 0)) == -1 and bind(p=(0, 0, 0x4000)) == -1
    assert bind(g=(0x1001, 0, 0x2000)) == -2 and bind(p=(0x3001, 0, 0x4000)) == -2
    assert bind(lr=(1.0, -1.0, 1.0)) == -1 and bind(wd=(1.0, 1.0, float("nan"))) == -1
    assert bind(image=None) == -1
    assert L.zero_multi_bind(None, None, None, None, None, image) == -1
    assert np.array_equal(host, before)                    # nothing written on error
    assert bind(lr=(1.0, 2.0, 0.5)) == 0                   # an empty tensor has no address
    empty = make(zf, [])[1]
    assert L.zero_multi_bind(C.byref(empty), None, None, None, None, None) == 0
    rc, plan32, host32 = make(zf, [4], param=-1)
    one = (C.c_void_p * 1)(0x1000)
    assert L.zero_multi_bind(C.byref(plan32), one, one, None, None,
                             C.c_void_p(host32.ctypes.data)) == -1


def test_calls_validate_before_launch(zf):
    L = zf.lib()
    hp = zf.zero_adamw_hparams_t(**HP)
    st = C.c_void_p(0x10000)
    for bits in (8, 32):
        rc, plan, host = make(zf, [300, 5], bits=bits)
        ref = C.byref(plan)
        sc = P if bits == 8 else None

        def step(d=P, p=P, m=P, v=P, ms=sc, vs=sc, hp=hp, flags=1, st=st, ref=ref):
            return L.zero_multi_adamw_step(ref, d, p, m, v, ms, vs,
                                           None if hp is None else C.byref(hp), 0, flags, st, None)

        assert step(ref=None) == -1 and step(d=None) == -1 and step(st=None) == -1
        assert step(hp=None) == -1 and step(flags=8) == -1 and step(flags=2) == -1
        assert step(d=C.c_void_p(0x1010)) == -2 and step(st=C.c_void_p(0x10004)) == -2
        assert step(p=None) == -1 and step(m=None) == -1 and step(v=None) == -1
        assert step(p=C.c_void_p(0x1008)) == -2 and step(m=C.c_void_p(0x1002)) == -2
        if bits == 8:
            assert step(ms=None) == -1 and step(vs=None) == -1
            assert step(vs=C.c_void_p(0x1002)) == -2
            assert step(hp=zf.zero_adamw_hparams_t(**dict(HP, eps=1e-40))) == -1
        bad = zf.zero_adamw_hparams_t(**dict(HP, beta2=1.0))
        assert step(hp=bad) == -1
        assert b"zero_multi_adamw_step" in L.zero_last_error()
        # the same call through the struct of its arguments
        assert L.zero_multi_adamw_step_args(None, None) == -1
        args = zf.zero_multi_step_args_t(C.addressof(plan), 0x1000, 0x1000, 0x1000, 0x1000,
                                         *[0x1000 if bits == 8 else None] * 2, None, hp, 0, 1)
        assert L.zero_multi_adamw_step_args(C.byref(args), None) == -1      # no state
        args.d_state, args.master = 0x10000, 0x1008
        assert L.zero_multi_adamw_step_args(C.byref(args), None) == -2
    assert L.zero_multi_unscale_norm(ref, None, 0, st, None) == -1
    assert L.zero_multi_unscale_norm(ref, P, 0, None, None) == -1
    assert L.zero_multi_unscale_norm(ref, P, 1, st, None) == -1
    assert L.zero_multi_unscale_norm(None, P, 0, st, None) == -1
    assert L.zero_multi_unscale_norm(ref, C.c_void_p(0x1080), 0, st, None) == -2
    blank = zf.zero_multi_plan_t()
    assert L.zero_multi_unscale_norm(C.byref(blank), P, 0, st, None) == -1
    rc, plan, host = make(zf, [300], bits=0, param=-1)
    assert L.zero_multi_adamw_step(C.byref(plan), P, P, P, P, None, None, C.byref(hp), 0, 1, st,
                                   None) == -1


def test_binding_refusals(zf):
    """The Python layer's own checks, on host tensors."""
    t = torch.zeros(8)
    with pytest.raises(ValueError, match="device"):
        zf.TensorListOptimizer([t], HP)
    with pytest.raises(ValueError, match="at least one"):
        zf.TensorListOptimizer([], HP)
    with pytest.raises(ValueError, match="grad_dtype"):
        zf.MultiPlan([8], torch.float64, device="cpu")
    with pytest.raises(ValueError, match="param_dtype"):
        zf.MultiPlan([8], torch.float32, torch.float32, device="cpu")
    with pytest.raises(zf.ZeroError):
        zf.MultiPlan([-8], torch.float32, device="cpu")
    plan = zf.MultiPlan([8, 9], torch.float16, device="cpu")
    with pytest.raises(RuntimeError, match="bind"):
        zf.zero_multi_unscale_norm(plan, None)
    with pytest.raises(ValueError, match="one entry per tensor"):
        plan.bind([torch.zeros(8, dtype=torch.float16)])
    with pytest.raises(ValueError, match="device"):
        plan.bind([torch.zeros(8, dtype=torch.float16), torch.zeros(9, dtype=torch.float16)])


def test_state_fields_are_views(zf):
    st = zf.StepState(1024.0, True, device="cpu")
    assert st.field("loss_scale").item() == 1024.0 and st.field("step").dtype == torch.int32
    st.field("sumsq").fill_(4.0)
    assert st.read().sumsq == 4.0
