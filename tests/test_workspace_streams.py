"""Which stream a call's own memory is taken under (no GPU needed).  torch's
allocator gives out a block again while the kernels that used it last are still
queued, and orders the new use behind them only on the stream that the block is
taken under: memory for kernels on another stream must be taken under that one."""
import contextlib

import pytest
import torch

CURRENT = 0x100


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


class Stream:
    def __init__(self, handle, name="stream"):
        self.cuda_stream, self.name, self.device = handle, name, torch.device("cuda", 0)


@pytest.fixture
def zf():
    import fsdp_sharded_mixed_flatparameter_amd as m
    return m


@pytest.fixture
def taken(zf, monkeypatch):
    """The streams under which memory was taken (None: the current one), and the
    library's launches as (name, stream) in place of the library."""
    under, log, real = [None], [], torch.empty

    @contextlib.contextmanager
    def on(stream):
        under.append((stream.name, stream.cuda_stream))
        yield
        under.pop()

    def empty(*size, device=None, **kw):
        log.append(("memory", under[-1]))
        return real(*size, **kw)

    class Library:
        def __getattr__(self, name):
            if name.endswith("_workspace"):
                return getattr(zf.lib(), name)

            def launch(*args):
                assert under == [None]
                log.append((name, args[-1]))
                return 0
            return launch

    monkeypatch.setattr(zf.unit, "_device", lambda: 0)
    monkeypatch.setattr(zf.unit, "_current_raw_stream", lambda: CURRENT)
    monkeypatch.setattr(zf.unit, "_lib", Library())
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: Stream(handle, "external"))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: Stream(0, "default"))
    monkeypatch.setattr(torch, "empty", empty)
    return log


class Handle:
    """Another library's stream object."""
    cuda_stream = 0x300


CASES = [(None, None, CURRENT), (Stream(CURRENT), None, CURRENT), (CURRENT, None, CURRENT),
         (Stream(0x200), ("stream", 0x200), 0x200), (0x200, ("external", 0x200), 0x200),
         (Handle(), ("external", 0x300), 0x300), (0, ("default", 0), 0), (1, ("default", 0), 1)]


@pytest.mark.parametrize("stream,under,handle", CASES)
def test_embed_grad(zf, taken, stream, under, handle):
    n, v, d = 5000, 70, 16
    tok, dy, g = (Device(torch.zeros(n, dtype=torch.int64), 1 << 24), Device(torch.zeros(n, d), 1 << 25),
                  Device(torch.zeros(v, d), 1 << 26))
    zf.zero_embed_grad(tok, dy, g, stream=stream)
    assert taken == [("memory", under), ("zero_embed_grad", handle)]


@pytest.mark.parametrize("stream,under,handle", CASES)
def test_weight_grad(zf, taken, stream, under, handle):
    s = zf.Saved8(5000, 40, device="cpu")
    s._at = (0, (1 << 24, (1 << 24) + s.codes.numel(), 1), (1 << 25, (1 << 25) + s.exponents.numel(), 1))
    taken.clear()
    dy, g = Device(torch.zeros(5000, 24, dtype=torch.bfloat16), 1 << 26), Device(torch.zeros(24, 40), 1 << 27)
    zf.zero_weight_grad8(dy, s, g, stream=stream)
    assert taken == [("memory", under), ("zero_weight_grad8", handle)]


@pytest.mark.parametrize("stream,under,handle", CASES)
@pytest.mark.parametrize("several", (False, True))
def test_an_optimizers_reduced_shard(zf, taken, monkeypatch, several, stream, under, handle):
    """The fp32 gradient shard that an optimizer takes at its first step."""
    monkeypatch.setattr(zf, "_current_raw_stream", lambda: CURRENT)
    real = torch.empty_like
    monkeypatch.setattr(torch, "empty_like", lambda t: torch.empty(0) if isinstance(t, Device) else real(t))
    master = Device(real(torch.zeros(64)), 1 << 24)
    if several:
        opt = object.__new__(zf.MultiShardOptimizer)
        opt.master, opt._red = [master, master], [None, None]
        a, b = opt._reduced(1, stream), opt._reduced(1, 0x400)
    else:
        opt = object.__new__(zf.ShardOptimizer)
        opt.master, opt._red = master, None
        a, b = opt.reduced_buffer(stream), opt.reduced_buffer(0x400)
    assert a is b and taken == [("memory", under)]
