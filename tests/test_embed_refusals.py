"""What the embedding's entry points refuse before anything is launched (no GPU
needed): the library on its arguments, and the binding on its tensors."""
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


def lookup(zf, tokens=P, token_bytes=8, n=4, first=0, table=P, tdt=2, vocab=10, dim=8, out=P, odt=2, ld=8):
    return zf.lib().zero_embed_lookup(tokens, token_bytes, n, first, table, tdt, vocab, dim, 1.0, out, odt, ld, None)


def lookup8(zf, n=4, q=P, s=P, n_slots=2, slot=40, block=256, offset=0, vocab=10, dim=8, ld=8):
    return zf.lib().zero_embed_lookup_int8(P, 8, n, 0, q, s, n_slots, slot, block, offset, vocab, dim, 1.0, P, 2,
                                           ld, None)


def grad(zf, tokens=P, token_bytes=8, n=4, first=0, dy=P, ddt=2, ld=8, g=P, gdt=2, vocab=10, dim=8, flags=0, ws=P,
         bytes_=1 << 40):
    return zf.lib().zero_embed_grad(tokens, token_bytes, n, first, None, dy, ddt, ld, 1.0, g, gdt, vocab, dim, flags,
                                    ws, bytes_, None)


@pytest.mark.parametrize("kw,code", [
    (dict(token_bytes=2), EINVAL), (dict(n=-1), EINVAL), (dict(first=-1), EINVAL), (dict(vocab=-1), EINVAL),
    (dict(dim=-1), EINVAL), (dict(n=(1 << 28) + 1), ERANGE), (dict(vocab=(1 << 25) + 1), ERANGE),
    (dict(dim=(1 << 24) + 1), ERANGE), (dict(tokens=None), EINVAL), (dict(tokens=at(0x10004)), EALIGN),
    (dict(tdt=7), EINVAL), (dict(odt=-1), EINVAL), (dict(table=None), EINVAL), (dict(table=at(0x10001)), EALIGN),
    (dict(out=None), EINVAL), (dict(out=at(0x10002), odt=0), EALIGN), (dict(ld=7), EINVAL),
    (dict(n=1 << 28, ld=1 << 40), ERANGE)])
def test_lookup_refuses(zf, kw, code):
    assert lookup(zf, **kw) == code
    assert zf.lib().zero_last_error().decode().startswith("zero_embed_lookup: ")


@pytest.mark.parametrize("kw,code", [
    (dict(block=128), EINVAL), (dict(n_slots=0), ERANGE), (dict(n_slots=65537), ERANGE), (dict(slot=-1), EINVAL),
    (dict(offset=-1), EINVAL), (dict(offset=1), EINVAL), (dict(slot=39), EINVAL), (dict(slot=1 << 62), ERANGE),
    (dict(offset=(1 << 63) - 1), ERANGE), (dict(q=None), EINVAL), (dict(s=None), EINVAL),
    (dict(s=at(0x10002)), EALIGN), (dict(ld=7), EINVAL)])
def test_lookup_in_the_payload_refuses(zf, kw, code):
    assert lookup8(zf, **kw) == code
    assert zf.lib().zero_last_error().decode().startswith("zero_embed_lookup_int8: ")


@pytest.mark.parametrize("kw,code", [
    (dict(token_bytes=0), EINVAL), (dict(n=-1), EINVAL), (dict(tokens=None), EINVAL), (dict(ddt=3), EINVAL),
    (dict(gdt=9), EINVAL), (dict(ld=-1), EINVAL), (dict(n=1 << 28, ld=1 << 40), ERANGE), (dict(flags=1), EINVAL),
    (dict(dy=None), EINVAL), (dict(g=None), EINVAL), (dict(dy=at(0x10001)), EALIGN), (dict(g=at(0x10002), gdt=0), EALIGN),
    (dict(n=1 << 28, dim=1 << 14, ld=0, bytes_=1 << 62), ERANGE), (dict(n=5000, ws=None), EINVAL), (dict(n=5000, bytes_=100), EINVAL), (dict(n=5000, ws=at(0x10008)), EALIGN)])
def test_grad_refuses(zf, kw, code):
    assert grad(zf, **kw) == code
    assert zf.lib().zero_last_error().decode().startswith("zero_embed_grad: ")


def test_calls_with_nothing_to_do(zf):
    assert lookup(zf, n=0, tokens=None, table=None, out=None) == 0
    assert lookup(zf, dim=0, table=None, out=None) == 0
    assert lookup8(zf, n=0, q=None, s=None) == 0
    assert grad(zf, n=0, tokens=None, dy=None, g=None, ws=None, bytes_=0, flags=8) == 0
    assert grad(zf, vocab=0, dy=None, g=None, ws=None, bytes_=0) == 0
    assert grad(zf, dim=0, dy=None, g=None, ws=None, bytes_=0) == 0


def test_workspace_size(zf):
    assert zf.zero_embed_grad_workspace(0, 0, 0) >= 0
    # keys and places twice, a byte per row, two fp32 rows per tile
    n, v, d = 100000, 5000, 1000
    assert 16 * n + v + 2 * (n // 128) * d * 4 <= zf.zero_embed_grad_workspace(n, v, d) <= 18 * n + v + 2 * (n // 128 + 2) * d * 4
    with pytest.raises(zf.ZeroError):
        zf.zero_embed_grad_workspace(-1, 5, 5)
    with pytest.raises(zf.ZeroError):
        zf.zero_embed_grad_workspace(1, 1 << 26, 5)


def test_host_tensors_are_refused(zf):
    tok, w, y = torch.zeros(4, dtype=torch.int64), torch.zeros(10, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device"):
        zf.zero_embed_lookup(tok, w, y)
    with pytest.raises(ValueError, match="device"):
        zf.zero_embed_grad(tok, y, w)
    with pytest.raises(ValueError, match="device"):
        zf.zero_embed_lookup_int8(tok, torch.zeros(80, dtype=torch.int8), torch.zeros(1), 1, 80, 0, 10, y)


def test_other_types_are_refused(zf):
    tok, w, y = torch.zeros(4), torch.zeros(10, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="tokens must be int64 or int32"):
        zf.zero_embed_lookup(tok, w, y)


class Device:
    """Stands for a device tensor, of which the checks ask shape, type and place only."""

    def __init__(self, t, index=0, base=1 << 20):
        self.t, self.base = t, base
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index

    def __getattr__(self, name):
        return getattr(self.t, name)

    def data_ptr(self):
        return self.base + self.t.storage_offset() * self.t.element_size()


def test_another_device_is_refused(zf, monkeypatch):
    monkeypatch.setattr(zf.unit, "_device", lambda: 0)
    u, f = zf.unit, zf.unit._FLOATS
    with pytest.raises(ValueError, match="x is on cuda:1, the current device is cuda:0"):
        u._flat(Device(torch.zeros(4), index=1), "x", f, 0)
    with pytest.raises(ValueError, match="x is on cuda:1"):
        u._rows(Device(torch.zeros(4, 2), index=1), "x", 4, 2, f, 0)
    assert u._flat(Device(torch.zeros(4)), "x", f, 0) == (1 << 20, (1 << 20) + 16, 0)


def test_rows_and_overlaps(zf):
    u, f = zf.unit, zf.unit._FLOATS
    t = torch.zeros(6, 20)

    def rows(t, n, cols, written=False):
        return u._rows(Device(t), "x", n, cols, f, 0, written)

    base = 1 << 20
    assert rows(t, 6, 20) == (base, base + 480, 0, 20)
    assert rows(t[:, 3:9], 6, 6) == (base + 12, base + 12 + 4 * 106, 0, 20)
    assert rows(t[0].expand(6, 20), 6, 20) == (base, base + 80, 0, 0)
    assert rows(t.view(2, 3, 20), 6, 20)[3] == 20
    assert rows(t[:1, 3:9], 1, 6, True) == (base + 12, base + 36, 0, 6)
    assert rows(t[:0], 0, 20)[3] == 20
    for bad, n, cols, written in ((t, 6, 19, False), (t, 5, 20, False), (t[:, ::2], 6, 10, False),
                                  (t.t(), 20, 6, False), (t[0].expand(6, 20), 6, 20, True),
                                  (t.view(2, 3, 20)[:, :, :5], 6, 5, False), (t[0, 0], 1, 1, False)):
        with pytest.raises(ValueError, match="x must"):
            rows(bad, n, cols, written)

    def apart(a, b):
        u._apart(rows(a, *a.shape), rows(b, *b.shape), "a", "b")

    apart(t[:, :8], t[:, 8:])
    apart(t[:, 8:], t[:, :8])
    apart(t[:, 8:9], t[:, 9:])
    apart(t[:3], t[3:])
    apart(t[:0], t)
    for a, b in ((t, t), (t[:, :8], t[:, 7:]), (t[:, 7:], t[:, :8]), (t[1:, :8], t[:-1, 4:12]), (t[:4], t[3:]),
                 (t[:, 2:5], t[2])):
        with pytest.raises(ValueError, match="a and b overlap"):
            apart(a, b if b.dim() == 2 else b[None])


def test_numbers_that_the_library_could_not_hold_are_refused(zf, monkeypatch):
    """A Python number past the library's integers must not arrive as another one."""
    monkeypatch.setattr(zf.unit, "_device", lambda: 0)
    tok, w, y = Device(torch.zeros(4, dtype=torch.int64)), Device(torch.zeros(10, 8), 0, 1 << 21), \
        Device(torch.zeros(4, 8), 0, 1 << 22)
    q, s = Device(torch.zeros(80, dtype=torch.int8), 0, 1 << 23), Device(torch.zeros(1), 0, 1 << 24)
    monkeypatch.setattr(zf.unit, "_lib", None)
    for first in (1 << 64, -(1 << 64) + 3, 1 << 63):
        with pytest.raises(ValueError, match="first"):
            zf.zero_embed_lookup(tok, w, y, first=first)
        with pytest.raises(ValueError, match="first"):
            zf.zero_embed_grad(tok, y, w, first=first)
        with pytest.raises(ValueError, match="first"):
            zf.zero_embed_lookup_int8(tok, q, s, 1, 80, 0, 10, y, first=first)
        with pytest.raises(ValueError, match="padding"):
            zf.zero_embed_grad(tok, y, w, padding=first)
    good = dict(n_slots=1, slot_numel=80, elem_offset=0, vocab=10, block=256)
    for name, value in (("n_slots", 1 << 32), ("n_slots", -(1 << 32) + 1), ("slot_numel", -(1 << 64) + 80),
                        ("elem_offset", 1 << 64), ("vocab", (1 << 64) + 10), ("block", 0), ("block", (1 << 32) + 256)):
        kw = {**good, name: value}
        if name == "n_slots":
            kw["slot_numel"] = 0
        with pytest.raises(ValueError, match=name):
            zf.zero_embed_lookup_int8(tok, q, s, out=y, **kw)


def test_a_workspace_that_overlaps_is_refused(zf, monkeypatch):
    monkeypatch.setattr(zf.unit, "_device", lambda: 0)
    monkeypatch.setattr(zf.unit, "_current_raw_stream", lambda: 0)
    n, v, d = 5000, 700, 16
    need = zf.zero_embed_grad_workspace(n, v, d)
    assert need > 0
    tok, dy, g = (Device(torch.zeros(n, dtype=torch.int64), 0, 1 << 24), Device(torch.zeros(n, d), 0, 1 << 25),
                  Device(torch.zeros(v, d), 0, 1 << 26))
    monkeypatch.setattr(zf.unit, "_lib", None)
    for other, name in ((tok, "tokens"), (dy, "dy"), (g, "grad")):
        ws = Device(torch.zeros(need, dtype=torch.uint8), 0, other.base - need + 1)
        with pytest.raises(ValueError, match="workspace and %s overlap" % name):
            zf.zero_embed_grad(tok, dy, g, workspace=ws)
