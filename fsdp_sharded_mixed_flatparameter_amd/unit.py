"""What a model's unit does between its gather and its reduce, next to the
library's step: rows of an embedding read from the gathered flat parameter (or
straight from the gathered INT8 payload), their gradient, summed by sorted
tokens into the flat gradient, activations kept in 8 bits, the functions that
keep and read them, and the weight gradient taken from them.  No arithmetic
happens here.

Every tensor of a call is on the current device, and so is its stream.  The calls
are ordered on the current stream, or on `stream`; tensors used on a stream other
than their own are ordered, and kept, by the caller; memory that a call takes for
itself belongs to the stream that it is ordered on.  Matrices are tensors whose
last dimension is contiguous: a row may be any distance from the next, so a slice
of columns needs no copy.
"""
import ctypes as C
import functools

import torch

from . import _DTYPE_CODES, _check, _current_raw_stream, _dtype_name, _lib, _stream, _torch_stream

ZERO_ACCUMULATE = 8
ZERO_GELU, ZERO_GELU_TANH, ZERO_SILU = 0, 1, 2
_KINDS = frozenset((ZERO_GELU, ZERO_GELU_TANH, ZERO_SILU))      # the library refuses the others
ZERO_BLOCK8 = 32                 # columns that share an exponent

# the checks below run before every launch, and a small call is as long as its
# host's part: tensors are asked once each, and details only for an error
_FLOATS = {getattr(torch, n): c for n, c in _DTYPE_CODES.items()}
_HALVES = {t: c for t, c in _FLOATS.items() if t != torch.float32}
_FP32, _INT8, _UINT8 = {torch.float32: 0}, {torch.int8: 1}, {torch.uint8: 1}
_TOKENS = {torch.int64: 8, torch.int32: 4}
_SIZE = (4, 2, 2)                # of the types' codes
_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _refuse(t, name, codes):
    """Says what is wrong with the type or the place of a tensor."""
    if t.dtype not in codes:
        raise ValueError("%s must be %s, not %s" % (name, " or ".join(_dtype_name(d) for d in codes), t.dtype))
    if t.get_device() < 0:
        raise ValueError("%s must be a device (CUDA) tensor" % name)
    raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, t.get_device(), _device()))


def _here(t, name, codes):
    """The current device, which `t` has to be on."""
    d = t.get_device()
    if d < 0 or t.dtype not in codes or d != _device():
        _refuse(t, name, codes)
    return d


def _flat(t, name, codes, here):
    """(first byte, byte behind the last, code of its type) of a contiguous argument."""
    code = codes.get(t.dtype)
    if code is None or t.get_device() != here:
        _refuse(t, name, codes)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    p = t.data_ptr()
    return p, p + t.nbytes, code


def _rows(t, name, rows, cols, codes, here, written=False):
    """(first byte, byte behind the last, code of its type, row distance) of a matrix
    argument: (rows, cols), or a contiguous tensor of that many elements whose last
    dimension is cols."""
    code = codes.get(t.dtype)
    if code is None or t.get_device() != here:
        _refuse(t, name, codes)
    shape = t.shape
    if shape != (rows, cols) and (not shape or shape[-1] != cols or t.numel() != rows * cols):
        raise ValueError("%s must hold %d rows of %d, not %s" % (name, rows, cols, tuple(shape)))
    p, size = t.data_ptr(), _SIZE[code]
    if t.is_contiguous():
        return p, p + rows * cols * size, code, cols
    ld, step = t.stride() if len(shape) == 2 else (0, 0)
    if len(shape) != 2 or (cols > 1 and step != 1) or (written and rows > 1 and ld < cols):
        raise ValueError("%s must be contiguous, or a matrix whose rows are" % name)
    ld = ld if rows > 1 else cols
    return p, p + ((rows - 1) * ld + cols) * size, code, ld


def _apart(a, b, name_a, name_b):
    """Refuses two arguments, as _flat and _rows give them, of which one is written
    where the other is used."""
    if a[0] >= b[1] or b[0] >= a[1] or a[0] == a[1] or b[0] == b[1]:
        return
    if len(a) == len(b) == 4 and a[2] == b[2] and a[3] == b[3] > 0:
        # columns of one buffer: the distance of the rows' beginnings, within a row
        size, ld = 2 if a[2] else 4, a[3]
        cols_a, cols_b = ((x[1] - x[0]) // size % ld or ld for x in (a, b))
        off = (b[0] - a[0]) // size % ld
        if cols_a <= off and off + cols_b <= ld and (b[0] - a[0]) % size == 0:
            return
    raise ValueError("%s and %s overlap" % (name_a, name_b))


_INT32 = (1 << 31) - 1


def _whole(x, name, most=(1 << 63) - 1):
    """Refuses a number that would arrive at the library as another one."""
    if not -most <= x <= most:
        raise ValueError("%s is out of range" % name)


def _on(stream):
    """The call's stream as an integer handle."""
    if stream is None:
        return _current_raw_stream()
    if isinstance(stream, torch.cuda.Stream) and stream.device.index != _device():
        raise ValueError("the stream is of cuda:%d, the current device is cuda:%d" % (stream.device.index, _device()))
    return _stream(stream).value or 0


def _scratch(workspace, need, device, here, stream, handle, used):
    """The call's workspace: the caller's, apart from the arguments in `used`, or one
    of the call's own.  torch's allocator orders the use of a block behind its last
    one on the stream that it is taken under, and on no other: the call's own is
    taken under the stream that its kernels go on."""
    if workspace is not None:
        w = _flat(workspace, "workspace", _UINT8, here)
        if workspace.numel() < need:
            raise ValueError("the workspace needs %d bytes" % need)
        for name, x in used:
            _apart(w, x, "workspace", name)
        return workspace
    if stream is None or handle == _current_raw_stream():
        return torch.empty(need, dtype=torch.uint8, device=device)
    with torch.cuda.stream(_torch_stream(stream, handle, here)):
        return torch.empty(need, dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ embedding
def _table(t, name, here):
    x = _flat(t, name, _FLOATS, here)
    if t.dim() != 2:
        raise ValueError("%s must be a matrix (rows by token)" % name)
    return x, t.shape


def zero_embed_lookup(tokens, table, out, scale=1.0, first=0, stream=None):
    """out[t] = table[tokens[t] - first] * scale, zeros for a token outside the
    table.  tokens: int32 or int64 of any shape; table: (vocab, dim), a view of
    the flat parameter; out: a row per token, fp32, fp16 or bf16."""
    _whole(first, "first")
    here = _here(tokens, "tokens", _TOKENS)
    t, n = _flat(tokens, "tokens", _TOKENS, here), tokens.numel()
    w, (vocab, dim) = _table(table, "table", here)
    y = _rows(out, "out", n, dim, _FLOATS, here, True)
    _apart(y, w, "out", "table")
    _apart(y, t, "out", "tokens")
    rc = _lib.zero_embed_lookup(t[0], t[2], n, first, w[0], w[2], vocab, dim, scale, y[0], y[2], y[3], _on(stream))
    if rc:
        _check(rc)


def zero_embed_lookup_int8(tokens, q_buf, q_scales, n_slots, slot_numel, elem_offset, vocab, out, scale=1.0,
                           first=0, block=256, stream=None):
    """zero_embed_lookup on a table that lies elem_offset elements into the flat
    parameter whose n_slots INT8 slots have been gathered (the payload that
    zero_dequant_allgather takes)."""
    if block != 256:
        raise ValueError("block must be 256")
    for x, name in ((first, "first"), (slot_numel, "slot_numel"), (elem_offset, "elem_offset"), (vocab, "vocab")):
        _whole(x, name)
    _whole(n_slots, "n_slots", _INT32)
    here = _here(tokens, "tokens", _TOKENS)
    t, n = _flat(tokens, "tokens", _TOKENS, here), tokens.numel()
    q, s = _flat(q_buf, "q_buf", _INT8, here), _flat(q_scales, "q_scales", _FP32, here)
    if out.dim() == 0:
        raise ValueError("out must have a row per token")
    dim = out.shape[-1]
    y = _rows(out, "out", n, dim, _FLOATS, here, True)
    if q_buf.numel() < n_slots * slot_numel or q_scales.numel() < n_slots * -(-slot_numel // block):
        raise ValueError("buffers are shorter than n_slots slots")
    _apart(y, t, "out", "tokens")
    _apart(y, q, "out", "q_buf")
    _apart(y, s, "out", "q_scales")
    rc = _lib.zero_embed_lookup_int8(t[0], t[2], n, first, q[0], s[0], n_slots, slot_numel, block, elem_offset, vocab,
                                     dim, scale, y[0], y[2], y[3], _on(stream))
    if rc:
        _check(rc)


@functools.lru_cache(maxsize=256)
def zero_embed_grad_workspace(n_tokens, vocab, dim):
    """The bytes of workspace that zero_embed_grad needs (0 for few tokens)."""
    for x, name in ((n_tokens, "n_tokens"), (vocab, "vocab"), (dim, "dim")):
        _whole(x, name)
    b = C.c_int64(0)
    _check(_lib.zero_embed_grad_workspace(n_tokens, vocab, dim, C.byref(b)))
    return b.value


def zero_embed_grad(tokens, dy, grad, scale=1.0, first=0, padding=None, accumulate=False, workspace=None,
                    stream=None):
    """grad[v] = scale * the sum of dy's rows at the tokens first + v, every row
    written; with `accumulate`, added to what grad's rows hold.  Rows of dy at
    the token `padding` and at tokens outside grad take no part.  grad: (vocab,
    dim), a view of the flat gradient.  The result does not depend on the order
    in which the GPU does the work.  Without a workspace the call takes one of
    its own from torch's allocator; a captured graph that brings its own must
    not share it with what may run at the same time."""
    _whole(first, "first")
    if padding is not None:
        _whole(padding, "padding")
    here = _here(tokens, "tokens", _TOKENS)
    t, n = _flat(tokens, "tokens", _TOKENS, here), tokens.numel()
    g, (vocab, dim) = _table(grad, "grad", here)
    d = _rows(dy, "dy", n, dim, _FLOATS, here)
    _apart(g, d, "grad", "dy")
    _apart(g, t, "grad", "tokens")
    handle, ws, size = _on(stream), None, 0
    need = zero_embed_grad_workspace(n, vocab, dim)
    if need or workspace is not None:
        ws = _scratch(workspace, need, grad.device, here, stream, handle, (("tokens", t), ("dy", d), ("grad", g)))
        ws, size = ws.data_ptr(), ws.numel()
    pad = None if padding is None else C.byref(C.c_int64(padding))
    rc = _lib.zero_embed_grad(t[0], t[2], n, first, pad, d[0], d[2], d[3], scale, g[0], g[2], vocab, dim,
                              ZERO_ACCUMULATE if accumulate else 0, ws, size, handle)
    if rc:
        _check(rc)


# ------------------------------------------------------------------ activations in 8 bits
class Saved8:
    """The checkpoint of a (rows, cols) matrix in 8 bits: `codes` (rows, pitch) int8,
    pitch the columns rounded up to blocks of 32, and `exponents` (rows, pitch / 32)
    uint8.  A value stands for code * 2^(exponent - 133), NaN in a block whose
    exponent is 255.  The memory is uninitialised until a call fills it; both tensors
    stay where they are, and are loaded by copying into them."""

    __slots__ = ("_rows", "_cols", "_codes", "_exponents", "_at")

    def __init__(self, rows, cols, device="cuda"):
        rows, cols = int(rows), int(cols)
        if rows < 0 or cols < 0:
            raise ValueError("negative size")
        blocks = -(-cols // ZERO_BLOCK8)
        self._hold(rows, cols, torch.empty(rows, blocks * ZERO_BLOCK8, dtype=torch.int8, device=device),
                   torch.empty(rows, blocks, dtype=torch.uint8, device=device))

    def _hold(self, rows, cols, codes, exponents):
        self._rows, self._cols, self._codes, self._exponents = rows, cols, codes, exponents
        # device, codes and exponents as _flat gives them
        c, e = codes.data_ptr(), exponents.data_ptr()
        self._at = (codes.get_device(), (c, c + codes.numel(), 1), (e, e + exponents.numel(), 1))

    def __reduce__(self):
        # a copy, or one loaded from bytes, must ask its own tensors where they are
        return _held, (self._rows, self._cols, self._codes, self._exponents)

    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    codes = property(lambda self: self._codes)
    exponents = property(lambda self: self._exponents)


def _held(*parts):
    s = Saved8.__new__(Saved8)
    s._hold(*parts)
    return s


_NONE = (None, None, None)


def _saved(s, name, here=None, rows=None, cols=None):
    """(device, codes, exponents) of a checkpoint argument."""
    if s is None:
        return _NONE
    if rows is not None and (s._rows != rows or s._cols != cols):
        raise ValueError("%s is of a (%d, %d) matrix, not (%d, %d)" % (name, s._rows, s._cols, rows, cols))
    at = s._at
    if at[0] != here and (here is not None or at[0] < 0 or at[0] != _device()):
        _refuse(s._codes, name, _INT8)
    return at


def _at(x):
    return None if x is None else x[0]


def _apart_all(written, read, same=()):
    """Refuses overlaps of what is written with one another and with what is read,
    but for the pairs in `same`, which may be one and the same matrix.  Arguments
    are (name, what _flat or _rows gave, or None)."""
    for k, (name_a, a) in enumerate(written):
        if a is None:
            continue
        first, last = a[0], a[1]
        for other in (written[k + 1:], read):
            for name_b, b in other:
                if b is not None and first < b[1] and b[0] < last and not ((name_a, name_b) in same and a == b):
                    _apart(a, b, name_a, name_b)


def _parts(name, s):
    return [] if s is _NONE else [(name + ".codes", s[1]), (name + ".exponents", s[2])]


def zero_act_save8(x, saved, stream=None):
    """The checkpoint of x, a (saved._rows, saved._cols) matrix."""
    here, c, e = _saved(saved, "saved")
    m = _rows(x, "x", saved._rows, saved._cols, _FLOATS, here)
    _apart(c, m, "saved.codes", "x")
    _apart(e, m, "saved.exponents", "x")
    rc = _lib.zero_act_save8(m[0], m[2], saved._rows, saved._cols, m[3], c[0], e[0], _on(stream))
    if rc:
        _check(rc)


def zero_act_restore8(saved, out, stream=None):
    """out = the values that the checkpoint stands for, in out's type."""
    here, c, e = _saved(saved, "saved")
    m = _rows(out, "out", saved._rows, saved._cols, _FLOATS, here, True)
    _apart(m, c, "out", "saved.codes")
    _apart(m, e, "out", "saved.exponents")
    rc = _lib.zero_act_restore8(c[0], e[0], saved._rows, saved._cols, m[0], m[2], m[3], _on(stream))
    if rc:
        _check(rc)


def zero_act_forward8(kind, x, out, saved, up=None, saved_up=None, stream=None):
    """out = act(x), times `up` where that is given, and the checkpoints of x and up,
    in one pass.  kind: ZERO_GELU, ZERO_GELU_TANH or ZERO_SILU.  x and up may be
    columns of one buffer; out may be x or up itself."""
    if kind not in _KINDS:
        _whole(kind, "kind", _INT32)
    if (up is None) != (saved_up is None):
        raise ValueError("up and saved_up go together")
    rows, cols = saved._rows, saved._cols
    s = _saved(saved, "saved")
    here = s[0]
    su = _saved(saved_up, "saved_up", here, rows, cols)
    m = _rows(x, "x", rows, cols, _FLOATS, here)
    dt = {x.dtype: m[2]}
    y = _rows(out, "out", rows, cols, dt, here, True)
    u = None if up is None else _rows(up, "up", rows, cols, dt, here)
    _apart_all([("out", y)] + _parts("saved", s) + _parts("saved_up", su), [("x", m), ("up", u)],
               (("out", "x"), ("out", "up")))
    rc = _lib.zero_act_forward8(kind, m[0], m[3], _at(u), 0 if u is None else u[3], m[2], rows, cols, y[0], y[3],
                                s[1][0], s[2][0], _at(su[1]), _at(su[2]), _on(stream))
    if rc:
        _check(rc)


def zero_act_backward8(kind, dy, saved, dx, saved_up=None, dup=None, again=None, stream=None):
    """From the checkpoints of x and up: dx = dy * act'(x), times up where there is
    one, and dup = dy * act(x).  `again` takes the checkpoint of act(x), times up:
    the next layer's input for its weight gradient, which was not kept.  dx or dup
    may be dy itself."""
    if kind not in _KINDS:
        _whole(kind, "kind", _INT32)
    if (dup is None) != (saved_up is None):
        raise ValueError("dup and saved_up go together")
    rows, cols = saved._rows, saved._cols
    s = _saved(saved, "saved")
    here = s[0]
    su = _saved(saved_up, "saved_up", here, rows, cols)
    sa = _saved(again, "again", here, rows, cols)
    d = _rows(dy, "dy", rows, cols, _FLOATS, here)
    dt = {dy.dtype: d[2]}
    x = _rows(dx, "dx", rows, cols, dt, here, True)
    u = None if dup is None else _rows(dup, "dup", rows, cols, dt, here, True)
    _apart_all([("dx", x), ("dup", u)] + _parts("again", sa),
               [("dy", d)] + _parts("saved", s) + _parts("saved_up", su), (("dx", "dy"), ("dup", "dy")))
    rc = _lib.zero_act_backward8(kind, d[0], d[3], d[2], rows, cols, s[1][0], s[2][0], _at(su[1]), _at(su[2]), x[0], x[3],
                                 _at(u), 0 if u is None else u[3], _at(sa[1]), _at(sa[2]), _on(stream))
    if rc:
        _check(rc)


@functools.lru_cache(maxsize=256)
def zero_weight_grad8_workspace(rows, outs, cols):
    """The bytes of workspace that zero_weight_grad8 needs (0 where it does not split
    its sums)."""
    for x, name in ((rows, "rows"), (outs, "outs"), (cols, "cols")):
        _whole(x, name)
    b = C.c_int64(0)
    _check(_lib.zero_weight_grad8_workspace(rows, outs, cols, C.byref(b)))
    return b.value


def zero_weight_grad8(dy, saved, grad, accumulate=False, workspace=None, stream=None):
    """grad = dy^T x, the gradient of a linear layer's (outs, cols) weight from the
    checkpoint of its input; with `accumulate` added to what grad holds.  dy: (rows,
    outs), fp16 or bf16 (an fp32 dy is rounded by the caller, who knows its range);
    grad: a view of the flat gradient, fp32, fp16 or bf16.  The workspace is as
    zero_embed_grad's."""
    here, c, e = _saved(saved, "saved")
    g = _flat(grad, "grad", _FLOATS, here)
    if grad.dim() != 2 or grad.shape[1] != saved._cols:
        raise ValueError("grad must be a matrix of %d columns" % saved._cols)
    rows, cols, outs = saved._rows, saved._cols, grad.shape[0]
    d = _rows(dy, "dy", rows, outs, _HALVES, here)
    _apart(g, d, "grad", "dy")
    _apart(g, c, "grad", "saved.codes")
    _apart(g, e, "grad", "saved.exponents")
    handle = _on(stream)
    need, ws, size = zero_weight_grad8_workspace(rows, outs, cols), None, 0
    if need or workspace is not None:
        ws = _scratch(workspace, need, grad.device, here, stream, handle,
                      (("dy", d), ("grad", g), ("saved.codes", c), ("saved.exponents", e)))
        ws, size = ws.data_ptr(), ws.numel()
    rc = _lib.zero_weight_grad8(d[0], d[2], d[3], rows, outs, c[0], e[0], cols, g[0], g[2],
                                ZERO_ACCUMULATE if accumulate else 0, ws, size, handle)
    if rc:
        _check(rc)
