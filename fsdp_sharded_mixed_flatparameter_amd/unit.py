"""What a model's unit does between its gather and its reduce, next to the
library's step: rows of an embedding read from the gathered flat parameter (or
straight from the gathered INT8 payload), their gradient, summed by sorted
tokens into the flat gradient, activations kept in 8 bits, the functions that
keep and read them, and the weight gradient taken from them.  No arithmetic
happens here.

Every tensor of a call is on the current device.  The calls are ordered on the
current stream, or on `stream`; tensors used on a stream other than their own
are ordered, and kept, by the caller.  Matrices are tensors whose last
dimension is contiguous: a row may be any distance from the next, so a slice of
columns needs no copy.
"""
import ctypes as C

import torch

from . import (_FLOATS, _check, _current_raw_stream, _dtype_code, _dtype_name, _lib, _ptr, _stream)

ZERO_ACCUMULATE = 8
ZERO_GELU, ZERO_GELU_TANH, ZERO_SILU = 0, 1, 2
ZERO_BLOCK8 = 32                 # columns that share an exponent


def _here(t, name):
    """`t`, a tensor of the current device."""
    if not t.is_cuda:
        raise ValueError("%s must be a device (CUDA) tensor" % name)
    if t.device.index != torch.cuda.current_device():
        raise ValueError("%s is on %s, the current device is cuda:%d"
                         % (name, t.device, torch.cuda.current_device()))
    return t


def _typed(t, name, dtypes):
    if _dtype_name(t.dtype) not in dtypes:
        raise ValueError("%s must be %s, not %s" % (name, " or ".join(dtypes), t.dtype))
    return _here(t, name)


def _flat(t, name, dtypes):
    """A contiguous argument."""
    _typed(t, name, dtypes)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _rows(t, name, rows, cols, dtypes, written=False):
    """The row stride of a matrix argument: (rows, cols), or a contiguous tensor
    of that many elements whose last dimension is cols."""
    _typed(t, name, dtypes)
    if t.dim() == 0 or t.shape[-1] != cols or t.numel() != rows * cols:
        raise ValueError("%s must hold %d rows of %d, not %s" % (name, rows, cols, tuple(t.shape)))
    if t.is_contiguous() or t.numel() == 0:
        return cols
    if t.dim() != 2 or (cols > 1 and t.stride(1) != 1) or (written and rows > 1 and t.stride(0) < cols):
        raise ValueError("%s must be contiguous, or a matrix whose rows are" % name)
    return t.stride(0) if rows > 1 else cols


def _span(t):
    """[first, last) byte of a tensor's memory."""
    if t.numel() == 0:
        return 0, 0
    size = t.element_size()
    return t.data_ptr(), t.data_ptr() + (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))) * size


def _apart(a, b, name_a, name_b):
    """Refuses two tensors of which one is written where the other is used."""
    (a0, a1), (b0, b1) = _span(a), _span(b)
    if a1 <= b0 or b1 <= a0:
        return
    if a.dim() == 2 and b.dim() == 2 and a.element_size() == b.element_size() and a.stride(0) == b.stride(0) \
            and a.stride(1) == 1 and b.stride(1) == 1:
        # columns of one buffer: the distance of the rows' beginnings, within a row
        ld = a.stride(0)
        off = (b0 - a0) // a.element_size() % ld
        if a.shape[1] <= off and off + b.shape[1] <= ld and (b0 - a0) % a.element_size() == 0:
            return
    raise ValueError("%s and %s overlap" % (name_a, name_b))


def _scratch(workspace, need, device, stream):
    """The call's workspace: the caller's, or one of the call's own, which its
    stream keeps until the kernels are done with it."""
    if workspace is not None:
        _flat(workspace, "workspace", ("uint8",))
        if workspace.numel() < need:
            raise ValueError("the workspace needs %d bytes" % need)
        return workspace
    workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if stream is not None:
        s = _stream(stream).value or 0
        if s != _current_raw_stream():
            workspace.record_stream(stream if isinstance(stream, torch.cuda.Stream)
                                    else torch.cuda.ExternalStream(s))
    return workspace


# ------------------------------------------------------------------ embedding
def _tokens(tokens):
    _flat(tokens, "tokens", ("int64", "int32"))
    return _ptr(tokens), tokens.element_size(), tokens.numel()


def _table(t, name):
    _flat(t, name, _FLOATS)
    if t.dim() != 2:
        raise ValueError("%s must be a matrix (rows by token)" % name)
    return t.shape


def zero_embed_lookup(tokens, table, out, scale=1.0, first=0, stream=None):
    """out[t] = table[tokens[t] - first] * scale, zeros for a token outside the
    table.  tokens: int32 or int64 of any shape; table: (vocab, dim), a view of
    the flat parameter; out: a row per token, fp32, fp16 or bf16."""
    ptr, size, n = _tokens(tokens)
    vocab, dim = _table(table, "table")
    ld = _rows(out, "out", n, dim, _FLOATS, written=True)
    _apart(out, table, "out", "table")
    _apart(out, tokens, "out", "tokens")
    _check(_lib.zero_embed_lookup(ptr, size, n, first, _ptr(table), _dtype_code(table), vocab, dim, scale,
                                  _ptr(out), _dtype_code(out), ld, _stream(stream)))


def zero_embed_lookup_int8(tokens, q_buf, q_scales, n_slots, slot_numel, elem_offset, vocab, out, scale=1.0,
                           first=0, block=256, stream=None):
    """zero_embed_lookup on a table that lies elem_offset elements into the flat
    parameter whose n_slots INT8 slots have been gathered (the payload that
    zero_dequant_allgather takes)."""
    ptr, size, n = _tokens(tokens)
    _flat(q_buf, "q_buf", ("int8",))
    _flat(q_scales, "q_scales", ("float32",))
    if out.dim() == 0:
        raise ValueError("out must have a row per token")
    dim = out.shape[-1]
    ld = _rows(out, "out", n, dim, _FLOATS, written=True)
    if q_buf.numel() < n_slots * slot_numel or q_scales.numel() < n_slots * -(-slot_numel // block):
        raise ValueError("buffers are shorter than n_slots slots")
    for t, name in ((tokens, "tokens"), (q_buf, "q_buf"), (q_scales, "q_scales")):
        _apart(out, t, "out", name)
    _check(_lib.zero_embed_lookup_int8(ptr, size, n, first, _ptr(q_buf), _ptr(q_scales), n_slots, slot_numel,
                                       block, elem_offset, vocab, dim, scale, _ptr(out), _dtype_code(out), ld,
                                       _stream(stream)))


def zero_embed_grad_workspace(n_tokens, vocab, dim):
    """The bytes of workspace that zero_embed_grad needs."""
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
    ptr, size, n = _tokens(tokens)
    vocab, dim = _table(grad, "grad")
    ld = _rows(dy, "dy", n, dim, _FLOATS)
    _apart(grad, dy, "grad", "dy")
    _apart(grad, tokens, "grad", "tokens")
    workspace = _scratch(workspace, zero_embed_grad_workspace(n, vocab, dim), grad.device, stream)
    pad = None if padding is None else C.byref(C.c_int64(padding))
    _check(_lib.zero_embed_grad(ptr, size, n, first, pad, _ptr(dy), _dtype_code(dy), ld, scale, _ptr(grad),
                                _dtype_code(grad), vocab, dim, ZERO_ACCUMULATE if accumulate else 0,
                                _ptr(workspace), workspace.numel(), _stream(stream)))


# ------------------------------------------------------------------ activations in 8 bits
class Saved8:
    """The checkpoint of a (rows, cols) matrix in 8 bits: `codes` (rows, pitch) int8,
    pitch the columns rounded up to blocks of 32, and `exponents` (rows, pitch / 32)
    uint8.  A value stands for code * 2^(exponent - 133), NaN in a block whose
    exponent is 255.  The memory is uninitialised until a call fills it."""

    def __init__(self, rows, cols, device="cuda"):
        rows, cols = int(rows), int(cols)
        if rows < 0 or cols < 0:
            raise ValueError("negative size")
        pitch = -(-cols // ZERO_BLOCK8) * ZERO_BLOCK8
        self.rows, self.cols = rows, cols
        self.codes = torch.empty(rows, pitch, dtype=torch.int8, device=device)
        self.exponents = torch.empty(rows, pitch // ZERO_BLOCK8, dtype=torch.uint8, device=device)

    def _tensors(self, name):
        pitch = -(-self.cols // ZERO_BLOCK8) * ZERO_BLOCK8
        for t, part, dt, shape in ((self.codes, "codes", "int8", (self.rows, pitch)),
                                   (self.exponents, "exponents", "uint8", (self.rows, pitch // ZERO_BLOCK8))):
            _flat(t, "%s.%s" % (name, part), (dt,))
            if t.shape != shape:
                raise ValueError("%s.%s must be %s" % (name, part, shape))
        return self.codes, self.exponents


def _saved(s, name):
    """(codes, exponents) pointers of a checkpoint argument, or of none."""
    if s is None:
        return None, None
    c, e = s._tensors(name)
    return _ptr(c), _ptr(e)


def _fits(s, name, rows, cols):
    if s is not None and (s.rows, s.cols) != (rows, cols):
        raise ValueError("%s is of a (%d, %d) matrix, not (%d, %d)" % (name, s.rows, s.cols, rows, cols))


def _same_place(a, b):
    return a.data_ptr() == b.data_ptr() and a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()


def _apart_all(written, read, same=()):
    """Refuses overlaps of what is written with one another and with what is read,
    but for the pairs in `same`, which may be one and the same tensor."""
    for k, (a, name_a) in enumerate(written):
        for b, name_b in written[k + 1:] + read:
            if a is None or b is None or ((name_a, name_b) in same and _same_place(a, b)):
                continue
            _apart(a, b, name_a, name_b)


def _parts(s, name):
    return [] if s is None else [(s.codes, name + ".codes"), (s.exponents, name + ".exponents")]


def zero_act_save8(x, saved, stream=None):
    """The checkpoint of x, a (saved.rows, saved.cols) matrix."""
    c, e = _saved(saved, "saved")
    ld = _rows(x, "x", saved.rows, saved.cols, _FLOATS)
    _apart_all(_parts(saved, "saved"), [(x, "x")])
    _check(_lib.zero_act_save8(_ptr(x), _dtype_code(x), saved.rows, saved.cols, ld, c, e, _stream(stream)))


def zero_act_restore8(saved, out, stream=None):
    """out = the values that the checkpoint stands for, in out's type."""
    c, e = _saved(saved, "saved")
    ld = _rows(out, "out", saved.rows, saved.cols, _FLOATS, written=True)
    _apart_all([(out, "out")], _parts(saved, "saved"))
    _check(_lib.zero_act_restore8(c, e, saved.rows, saved.cols, _ptr(out), _dtype_code(out), ld, _stream(stream)))


def zero_act_forward8(kind, x, out, saved, up=None, saved_up=None, stream=None):
    """out = act(x), times `up` where that is given, and the checkpoints of x and up,
    in one pass.  kind: ZERO_GELU, ZERO_GELU_TANH or ZERO_SILU.  x and up may be
    columns of one buffer; out may be x or up itself."""
    if (up is None) != (saved_up is None):
        raise ValueError("up and saved_up go together")
    c, e = _saved(saved, "saved")
    uc, ue = _saved(saved_up, "saved_up")
    rows, cols = saved.rows, saved.cols
    _fits(saved_up, "saved_up", rows, cols)
    dt = (_dtype_name(x.dtype),)
    x_ld = _rows(x, "x", rows, cols, _FLOATS)
    y_ld = _rows(out, "out", rows, cols, dt, written=True)
    u_ld = 0 if up is None else _rows(up, "up", rows, cols, dt)
    _apart_all([(out, "out")] + _parts(saved, "saved") + _parts(saved_up, "saved_up"), [(x, "x"), (up, "up")],
               (("out", "x"), ("out", "up")))
    _check(_lib.zero_act_forward8(kind, _ptr(x), x_ld, _ptr(up), u_ld, _dtype_code(x), rows, cols, _ptr(out), y_ld,
                                  c, e, uc, ue, _stream(stream)))


def zero_act_backward8(kind, dy, saved, dx, saved_up=None, dup=None, again=None, stream=None):
    """From the checkpoints of x and up: dx = dy * act'(x), times up where there is
    one, and dup = dy * act(x).  `again` takes the checkpoint of act(x), times up:
    the next layer's input for its weight gradient, which was not kept.  dx or dup
    may be dy itself."""
    if (dup is None) != (saved_up is None):
        raise ValueError("dup and saved_up go together")
    c, e = _saved(saved, "saved")
    uc, ue = _saved(saved_up, "saved_up")
    ac, ae = _saved(again, "again")
    rows, cols = saved.rows, saved.cols
    _fits(saved_up, "saved_up", rows, cols)
    _fits(again, "again", rows, cols)
    dt = (_dtype_name(dy.dtype),)
    d_ld = _rows(dy, "dy", rows, cols, _FLOATS)
    x_ld = _rows(dx, "dx", rows, cols, dt, written=True)
    u_ld = 0 if dup is None else _rows(dup, "dup", rows, cols, dt, written=True)
    _apart_all([(dx, "dx"), (dup, "dup")] + _parts(again, "again"),
               [(dy, "dy")] + _parts(saved, "saved") + _parts(saved_up, "saved_up"),
               (("dx", "dy"), ("dup", "dy")))
    _check(_lib.zero_act_backward8(kind, _ptr(dy), d_ld, _dtype_code(dy), rows, cols, c, e, uc, ue, _ptr(dx), x_ld,
                                   _ptr(dup), u_ld, ac, ae, _stream(stream)))


def zero_weight_grad8_workspace(rows, outs, cols):
    """The bytes of workspace that zero_weight_grad8 needs (0 for most sizes)."""
    b = C.c_int64(0)
    _check(_lib.zero_weight_grad8_workspace(rows, outs, cols, C.byref(b)))
    return b.value


def zero_weight_grad8(dy, saved, grad, accumulate=False, workspace=None, stream=None):
    """grad = dy^T x, the gradient of a linear layer's (outs, cols) weight from the
    checkpoint of its input; with `accumulate` added to what grad holds.  dy: (rows,
    outs), fp16 or bf16; grad: a view of the flat gradient, fp32, fp16 or bf16.
    The workspace is as zero_embed_grad's."""
    c, e = _saved(saved, "saved")
    _flat(grad, "grad", _FLOATS)
    if grad.dim() != 2 or grad.shape[1] != saved.cols:
        raise ValueError("grad must be a matrix of %d columns" % saved.cols)
    rows, cols, outs = saved.rows, saved.cols, grad.shape[0]
    ld = _rows(dy, "dy", rows, outs, ("float16", "bfloat16"))
    _apart_all([(grad, "grad")], [(dy, "dy")] + _parts(saved, "saved"))
    need = zero_weight_grad8_workspace(rows, outs, cols)
    if need or workspace is not None:
        workspace = _scratch(workspace, need, grad.device, stream)
    _check(_lib.zero_weight_grad8(_ptr(dy), _dtype_code(dy), ld, rows, outs, c, e, cols, _ptr(grad),
                                  _dtype_code(grad), ZERO_ACCUMULATE if accumulate else 0, _ptr(workspace),
                                  0 if workspace is None else workspace.numel(), _stream(stream)))
