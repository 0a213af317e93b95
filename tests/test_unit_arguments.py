"""Arguments of a unit's operators that must not arrive at the library as others
(no GPU needed)."""
import pytest
import torch


class Device:
    """Stands for a device tensor, of which the checks ask shape, type and place only."""

    def __init__(self, t, base):
        self.t, self.base, self.device = t, base, torch.device("cuda", 0)

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)

    def data_ptr(self):
        return self.base


@pytest.fixture
def zf(monkeypatch):
    """The binding on a device 0, with a library that must not be called."""
    import fsdp_sharded_mixed_flatparameter_amd as m
    monkeypatch.setattr(m.unit, "_device", lambda: 0)
    monkeypatch.setattr(m.unit, "_current_raw_stream", lambda: 0)
    monkeypatch.setattr(m.unit, "_lib", None)
    return m


def saved(zf, rows, cols, base):
    s = zf.Saved8(rows, cols, device="cpu")
    s._at = (0, (base, base + s.codes.numel(), 1), (base + (1 << 20), base + (1 << 20) + s.exponents.numel(), 1))
    return s


@pytest.mark.parametrize("kind", [1 << 32, (1 << 32) + 2, -(1 << 32), (1 << 64) + 1, 1 << 31])
def test_a_kind_past_32_bits_is_refused(zf, kind):
    """It would arrive as another function."""
    s, x, y = saved(zf, 4, 40, 1 << 22), Device(torch.zeros(4, 40), 1 << 24), Device(torch.zeros(4, 40), 1 << 25)
    with pytest.raises(ValueError, match="kind is out of range"):
        zf.zero_act_forward8(kind, x, y, s)
    with pytest.raises(ValueError, match="kind is out of range"):
        zf.zero_act_backward8(kind, x, s, y)


class Stream:
    cuda_stream = 0x200

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def test_a_stream_of_another_device_is_refused(zf, monkeypatch):
    """Kernels would run there on this device's memory."""
    class Library:
        def __getattr__(self, name):
            def launch(*args):
                raise RuntimeError("launched")
            return launch

    monkeypatch.setattr(zf.unit, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(zf.unit, "zero_embed_grad_workspace", lambda *a: 0)
    monkeypatch.setattr(zf.unit, "zero_weight_grad8_workspace", lambda *a: 0)
    s, x, y = saved(zf, 4, 40, 1 << 22), Device(torch.zeros(4, 40), 1 << 24), Device(torch.zeros(4, 40), 1 << 25)
    tok, half = Device(torch.zeros(4, dtype=torch.int64), 1 << 26), Device(torch.zeros(4, 4, dtype=torch.bfloat16), 1 << 27)
    q, scales = Device(torch.zeros(160, dtype=torch.int8), 1 << 28), Device(torch.zeros(1), 1 << 29)
    calls = [lambda st: zf.zero_embed_lookup(tok, x, y, stream=st),
             lambda st: zf.zero_embed_lookup_int8(tok, q, scales, 1, 160, 0, 4, y, stream=st),
             lambda st: zf.zero_embed_grad(tok, x, y, stream=st),
             lambda st: zf.zero_act_save8(x, s, stream=st), lambda st: zf.zero_act_restore8(s, y, stream=st),
             lambda st: zf.zero_act_forward8(zf.ZERO_SILU, x, y, s, stream=st),
             lambda st: zf.zero_act_backward8(zf.ZERO_SILU, x, s, y, stream=st),
             lambda st: zf.zero_weight_grad8(half, s, y, stream=st)]
    for call in calls:
        with pytest.raises(ValueError, match="the stream is of cuda:1, the current device is cuda:0"):
            call(Stream(1))
        with pytest.raises(RuntimeError, match="launched"):
            call(Stream(0))
