"""What the 8-bit activations' entry points refuse before anything is launched
(no GPU needed): the library on its arguments, and the binding on its tensors."""
import ctypes as C

import pytest
import torch

EINVAL, EALIGN, ERANGE = -1, -2, -3
P = C.c_void_p(0x10000)         # never dereferenced: validation fails first, or nothing is to be done


@pytest.fixture(scope="module")
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    return m


def at(x):
    return C.c_void_p(x)


def save(zf, x=P, dt=2, rows=4, cols=40, ld=40, q=P, e=P):
    return zf.lib().zero_act_save8(x, dt, rows, cols, ld, q, e, None)


def restore(zf, x=P, dt=2, rows=4, cols=40, ld=40, q=P, e=P):
    return zf.lib().zero_act_restore8(q, e, rows, cols, x, dt, ld, None)


MATRIX = [(dict(dt=3), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(cols=(1 << 24) + 1), ERANGE),
          (dict(rows=(1 << 40) + 1), ERANGE), (dict(x=None), EINVAL), (dict(x=at(0x10001)), EALIGN),
          (dict(x=at(0x10002), dt=0), EALIGN), (dict(ld=-1), EINVAL), (dict(rows=1 << 40, ld=1 << 30), ERANGE),
          (dict(q=None), EINVAL), (dict(e=None), EINVAL), (dict(q=at(0x10008)), EALIGN)]


@pytest.mark.parametrize("kw,code", MATRIX)
def test_save_and_restore_refuse(zf, kw, code):
    assert save(zf, **kw) == code and restore(zf, **kw) == code
    assert restore(zf, ld=39) == EINVAL


def forward(zf, kind=2, x=P, x_ld=40, up=None, u_ld=40, dt=2, rows=4, cols=40, y=P, y_ld=40, q=P, e=P, uq=None, ue=None):
    return zf.lib().zero_act_forward8(kind, x, x_ld, up, u_ld, dt, rows, cols, y, y_ld, q, e, uq, ue, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kind=3), EINVAL), (dict(kind=-1), EINVAL), (dict(dt=9), EINVAL), (dict(x=None), EINVAL), (dict(y=None), EINVAL),
    (dict(y_ld=39), EINVAL), (dict(x_ld=-1), EINVAL), (dict(q=None), EINVAL), (dict(up=P), EINVAL), (dict(up=P, uq=P), EINVAL),
    (dict(uq=P, ue=P), EINVAL), (dict(up=at(0x10001), uq=P, ue=P), EALIGN), (dict(up=P, uq=at(0x10004), ue=P), EALIGN),
    (dict(up=P, uq=P, ue=P, u_ld=-2), EINVAL)])
def test_forward_refuses(zf, kw, code):
    assert forward(zf, **kw) == code
    assert zf.lib().zero_last_error().decode().startswith("zero_act_forward8: ")


def backward(zf, kind=2, dy=P, d_ld=40, dt=2, rows=4, cols=40, q=P, e=P, uq=None, ue=None, dx=P, x_ld=40, dup=None,
             u_ld=40, aq=None, ae=None):
    return zf.lib().zero_act_backward8(kind, dy, d_ld, dt, rows, cols, q, e, uq, ue, dx, x_ld, dup, u_ld, aq, ae, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kind=5), EINVAL), (dict(dt=-1), EINVAL), (dict(dy=None), EINVAL), (dict(dx=None), EINVAL), (dict(x_ld=39), EINVAL),
    (dict(d_ld=-1), EINVAL), (dict(e=None), EINVAL), (dict(dup=P), EINVAL), (dict(uq=P, ue=P), EINVAL), (dict(uq=P, dup=P), EINVAL),
    (dict(uq=P, ue=P, dup=P, u_ld=39), EINVAL), (dict(aq=P), EINVAL), (dict(ae=P), EINVAL), (dict(aq=at(0x10001), ae=P), EALIGN),
    (dict(dx=at(0x10001)), EALIGN)])
def test_backward_refuses(zf, kw, code):
    assert backward(zf, **kw) == code
    assert zf.lib().zero_last_error().decode().startswith("zero_act_backward8: ")


def weight(zf, dy=P, dt=2, ld=24, rows=100, outs=24, q=P, e=P, cols=40, grad=P, gt=0, flags=0, ws=P, bytes_=1 << 40):
    return zf.lib().zero_weight_grad8(dy, dt, ld, rows, outs, q, e, cols, grad, gt, flags, ws, bytes_, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(gt=3), EINVAL), (dict(flags=1), EINVAL), (dict(rows=-1), EINVAL), (dict(outs=-1), EINVAL),
    (dict(cols=-1), EINVAL), (dict(rows=(1 << 36) + 1), ERANGE), (dict(cols=(1 << 24) + 1), ERANGE),
    (dict(outs=(1 << 24) + 1), ERANGE), (dict(outs=1 << 24, cols=1 << 24), ERANGE), (dict(grad=None), EINVAL),
    (dict(grad=at(0x10002)), EALIGN), (dict(dy=None), EINVAL), (dict(dy=at(0x10001)), EALIGN), (dict(ld=-1), EINVAL),
    (dict(q=None), EINVAL), (dict(q=at(0x10008)), EALIGN), (dict(rows=5000, ws=None), EINVAL),
    (dict(rows=5000, bytes_=100), EINVAL), (dict(rows=5000, ws=at(0x10004)), EALIGN)])
def test_weight_grad_refuses(zf, kw, code):
    assert weight(zf, **kw) == code
    assert zf.lib().zero_last_error().decode().startswith("zero_weight_grad8: ")


def test_calls_with_nothing_to_do(zf):
    for kw in (dict(rows=0), dict(cols=0)):
        assert save(zf, x=None, q=None, e=None, **kw) == 0
        assert restore(zf, x=None, q=None, e=None, **kw) == 0
        assert forward(zf, x=None, y=None, q=None, e=None, **kw) == 0
        assert backward(zf, dy=None, dx=None, q=None, e=None, **kw) == 0
    assert weight(zf, outs=0, grad=None) == 0 and weight(zf, cols=0, grad=None, q=None, e=None) == 0
    assert weight(zf, rows=0, dy=None, grad=None, q=None, e=None, flags=8) == 0


def test_workspace_sizes(zf):
    assert zf.zero_weight_grad8_workspace(2048, 4096, 4096) == 0         # a tile for every place of the chip
    assert zf.zero_weight_grad8_workspace(50, 64, 64) == 0               # rows too few to split
    need = zf.zero_weight_grad8_workspace(5000, 24, 40)
    assert need > 0 and need % (64 * 64 * 4) == 0                        # whole tiles' sums
    # the tiles behind the last full round are shared, the others are not
    need = zf.zero_weight_grad8_workspace(16384, 4099, 4001)
    assert 0 < need <= 16 * 96 * 256 * 256 * 4
    for bad in ((-1, 5, 5), (5, 1 << 25, 5)):
        with pytest.raises(zf.ZeroError):
            zf.zero_weight_grad8_workspace(*bad)


def test_tensors_are_refused(zf, monkeypatch):
    monkeypatch.setattr(zf.unit, "_device", lambda: 0)
    s = zf.Saved8(4, 40, device="cpu")
    assert s.codes.shape == (4, 64) and s.exponents.shape == (4, 2)
    x = torch.zeros(4, 40)
    with pytest.raises(ValueError, match="go together"):
        zf.zero_act_forward8(zf.ZERO_SILU, x, x, s, up=x)
    with pytest.raises(ValueError, match="saved must be a device"):
        zf.zero_act_save8(x, s)
    with pytest.raises(ValueError, match="go together"):
        zf.zero_act_backward8(zf.ZERO_SILU, x, s, x, dup=x)
    with pytest.raises(ValueError, match="negative"):
        zf.Saved8(-1, 4)


class Device:
    """Stands for a device tensor, of which the checks ask shape, type and place only."""

    def __init__(self, t, base):
        self.t, self.base, self.device = t, base, torch.device("cuda", 0)

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)

    def data_ptr(self):
        return self.base + self.t.storage_offset() * self.t.element_size()


@pytest.fixture
def place(zf, monkeypatch):
    """Tensors that pass for device tensors, and a library that must not be called."""
    monkeypatch.setattr(zf.unit, "_device", lambda: 0)
    monkeypatch.setattr(zf.unit, "_lib", None)
    base = [1 << 20]

    def make(*shape, dtype=torch.float32):
        base[0] += 1 << 20
        return Device(torch.zeros(*shape, dtype=dtype), base[0])

    def saved(rows, cols):
        s = zf.Saved8(rows, cols, device="cpu")
        base[0] += 2 << 20
        c, e = base[0] - (1 << 20), base[0]
        s._at = (0, (c, c + s.codes.numel(), 1), (e, e + s.exponents.numel(), 1))
        return s

    return make, saved


def test_shapes_and_overlaps_are_refused(zf, place):
    make, saved = place
    s, u, x, d = saved(4, 40), saved(4, 40), make(4, 40), make(4, 40)

    def refused(match, f, *a, **kw):
        with pytest.raises(ValueError, match=match):
            f(*a, **kw)

    refused("x must hold", zf.zero_act_save8, make(4, 41), s)
    refused("out must be float32", zf.zero_act_forward8, 0, x, make(4, 40, dtype=torch.float16), s)
    refused("saved_up is of", zf.zero_act_forward8, 0, x, d, s, up=x, saved_up=saved(4, 41))
    refused("overlap", zf.zero_act_forward8, 0, x, d, s, up=x, saved_up=s)
    shifted = Device(torch.zeros(5, 40)[1:], x.base)
    refused("overlap", zf.zero_act_forward8, 0, x, shifted, s)
    refused("dx and dup overlap", zf.zero_act_backward8, 0, d, s, x, saved_up=u, dup=x)
    refused("again.codes and saved.codes", zf.zero_act_backward8, 0, d, s, x, again=s)
    refused("again is of", zf.zero_act_backward8, 0, d, s, x, again=saved(5, 40))
    refused("grad must be a matrix", zf.zero_weight_grad8, make(4, 8, dtype=torch.bfloat16), s, make(8, 41))
    refused("dy must be float16", zf.zero_weight_grad8, make(4, 8), s, make(8, 40))
    refused("dy must hold", zf.zero_weight_grad8, make(4, 9, dtype=torch.bfloat16), s, make(8, 40))
    with pytest.raises(AttributeError):
        s.codes = torch.zeros(4, 40, dtype=torch.int8)      # a checkpoint's memory stays where it is


def test_a_copied_checkpoint_has_memory_of_its_own(zf):
    """Copies and what is loaded from bytes name their own tensors, never the first one's."""
    import copy
    import io
    import pickle
    s = zf.Saved8(4, 40, device="cpu")
    s.codes.copy_(torch.arange(256).view(4, 64) - 128)
    s.exponents.fill_(130)
    f = io.BytesIO()
    torch.save(s, f)
    f.seek(0)
    for c in (copy.deepcopy(s), pickle.loads(pickle.dumps(s)), torch.load(f, weights_only=False)):
        assert (c.rows, c.cols) == (4, 40) and torch.equal(c.codes, s.codes) and torch.equal(c.exponents, s.exponents)
        assert c.codes.data_ptr() != s.codes.data_ptr()
        assert c._at[1] == (c.codes.data_ptr(), c.codes.data_ptr() + 256, 1)
        assert c._at[2] == (c.exponents.data_ptr(), c.exponents.data_ptr() + 8, 1)
    c = copy.copy(s)
    assert c.codes is s.codes and c._at == s._at


def test_a_workspace_that_overlaps_is_refused(zf, place, monkeypatch):
    _, saved = place
    monkeypatch.setattr(zf.unit, "_current_raw_stream", lambda: 0)
    monkeypatch.setattr(zf.unit, "_lib", zf.lib())
    s = saved(5000, 40)
    need = zf.zero_weight_grad8_workspace(5000, 24, 40)
    assert need > 0
    dy, g = Device(torch.zeros(5000, 24, dtype=torch.bfloat16), 1 << 33), Device(torch.zeros(24, 40), 1 << 34)
    monkeypatch.setattr(zf.unit, "_lib", None)
    # the workspace's last byte is the argument's first; the exponents' last is the workspace's first
    for first, name in (((1 << 33) - need + 1, "dy"), ((1 << 34) - need + 1, "grad"),
                        (s._at[1][0] - need + 1, "saved.codes"), (s._at[2][1] - 1, "saved.exponents")):
        with pytest.raises(ValueError, match="workspace and %s overlap" % name):
            zf.zero_weight_grad8(dy, s, g, workspace=Device(torch.zeros(need, dtype=torch.uint8), first))
