"""What a model's unit does between its gather and its reduce, next to the
library's step: rows of an embedding read from the gathered flat parameter (or
straight from the gathered INT8 payload), and their gradient, summed by sorted
tokens into the flat gradient.  No arithmetic happens here.

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
