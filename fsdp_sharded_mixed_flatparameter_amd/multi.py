"""One rank's optimizer over a list of tensors: the plan that names them to the
library, and the optimizer that owns the state arenas and issues the calls of
one step.  No arithmetic happens here; the statistics and the step run in
libzeroflat.
"""
import ctypes as C
import itertools

import torch

from . import (_DTYPE_CODES, _FLOATS, ZERO_MULTI_STATISTICS, ZERO_NONE, ZERO_ROW,
               ZERO_STEP_FINALIZE, StepState, _check, _current_raw_stream, _dev, _dtype_name, _lib, _stream,
               zero_adamw_hparams_t, zero_multi_plan_t, zero_multi_step_args_t)


def _doubles(x, n, name):
    if x is None:
        return None
    x = [float(v) for v in x]
    if len(x) != n:
        raise ValueError("%s must have one entry per tensor (%d)" % (name, n))
    return (C.c_double * max(n, 1))(*x)


class MultiPlan:
    """The tables and the workspace of a list of tensors, on the device.

    `numels` and the dtypes are fixed; bind() names the tensors and may be called
    again whenever they move.  The plan keeps the tensors alive.  A plan is used
    by one stream at a time.  tensor_sumsq is a device view (fp64, one entry per
    tensor) of what the latest statistics wrote."""

    def __init__(self, numels, grad_dtype, param_dtype=None, state_bits=0, device="cuda"):
        numels = [int(x) for x in numels]
        n = len(numels)
        gname = _dtype_name(grad_dtype)
        pname = None if param_dtype is None else _dtype_name(param_dtype)
        if gname not in _FLOATS:
            raise ValueError("grad_dtype must be %s" % " or ".join(_FLOATS))
        if pname not in (None, "float16", "bfloat16"):
            raise ValueError("param_dtype must be float16 or bfloat16, or None")
        self.numels, self.grad_dtype, self.param_dtype = numels, grad_dtype, param_dtype
        self.state_bits = state_bits
        self._plan = zero_multi_plan_t()
        self._ref = C.byref(self._plan)
        arr = (C.c_int64 * max(n, 1))(*numels)
        args = (arr, n, _DTYPE_CODES[gname], ZERO_NONE if pname is None else _DTYPE_CODES[pname],
                state_bits, self._ref)
        _check(_lib.zero_multi_plan_init(*args, None, 0))
        self.rows = self._plan.rows
        host = torch.empty(self._plan.image_bytes, dtype=torch.uint8)
        _check(_lib.zero_multi_plan_init(*args, C.c_void_p(host.data_ptr()), host.numel()))
        self._image = host.to(device)
        self._image_ptr = C.c_void_p(self._image.data_ptr())
        self._entries = host[:self._plan.bind_bytes].clone()
        off = self._plan.sumsq_off
        self.tensor_sumsq = self._image[off:off + 8 * n].view(torch.float64)
        self._grads = self._params = None
        self._bound = n == 0

    def __len__(self):
        return len(self.numels)

    def _require_bound(self):
        if not self._bound:
            raise RuntimeError("the plan names no tensors yet: call bind first")

    def _tensors(self, tensors, name, dtype):
        tensors = list(tensors)
        if len(tensors) != len(self):
            raise ValueError("%s must have one entry per tensor (%d)" % (name, len(self)))
        dev, ptrs = self._image.device, []
        for k, (t, n) in enumerate(zip(tensors, self.numels)):
            if not (t.dtype == dtype and t.numel() == n and t.is_cuda and t.device == dev
                    and t.is_contiguous()):
                _dev(t, "%s[%d]" % (name, k), (_dtype_name(dtype),))
                if t.numel() != n:
                    raise ValueError("%s[%d] has %d elements, the plan says %d" % (name, k, t.numel(), n))
                raise ValueError("%s[%d] is on %s, the plan on %s" % (name, k, t.device, dev))
            ptrs.append(t.data_ptr() or None)
        return tensors, (C.c_void_p * max(len(self), 1))(*ptrs)

    def bind(self, grads, params=None, lr_mult=None, decay_mult=None):
        """Name the gradients, and the 16-bit parameters if the plan has them,
        with a learning-rate and a decay factor per tensor (all ones when not
        given).  Copies the table to the device and waits for the device before
        and after, so no step in flight sees half of it; not during capture.

        A step reads the memory named here, which the plan keeps alive, and not
        what a parameter's .grad is later: where backward allocates gradients
        anew (zero_grad(set_to_none=True)), a step without a new bind repeats
        the last gradients.  Zero them in place, or bind before every step (30 us
        of the host's time for 4 tensors, 200 us for 290, and the device is idle
        meanwhile)."""
        grads, g = self._tensors(grads, "grads", self.grad_dtype)
        p = None
        if self.param_dtype is None:
            if params is not None:
                raise ValueError("the plan has no param_dtype")
        elif params is None:
            raise ValueError("the plan has a param_dtype: params are needed")
        else:
            params, p = self._tensors(params, "params", self.param_dtype)
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("bind copies from the host: not during graph capture")
        _check(_lib.zero_multi_bind(self._ref, g, p, _doubles(lr_mult, len(self), "lr_mult"),
                                    _doubles(decay_mult, len(self), "decay_mult"),
                                    C.c_void_p(self._entries.data_ptr())))
        if len(self):
            torch.cuda.synchronize(self._image.device)
            self._image[:self._plan.bind_bytes].copy_(self._entries)
            torch.cuda.synchronize(self._image.device)
        self._grads, self._params, self._bound = grads, params, True


class TensorListOptimizer:
    """AdamW over a list of tensors with one step state: one norm, clip, skip
    and loss scale over all of them, and a learning-rate and decay factor each.

    master, exp_avg and exp_avg_sq are arenas of rows of 256 elements, tensor k
    from row first_row[k] on (views() gives the tensors inside one); the
    constructor copies `masters` into the first.  With state_bits 8, exp_avg is
    e4m3 and exp_avg_sq e5m2, with one scale per row in exp_avg_scale and
    exp_avg_sq_scale (None otherwise), and `seed` fixes the second moment's
    random rounding (seed s rounds at step t as s + 1 does at t - 1: give lists
    that train together seeds further apart than their steps).  The arenas stay where they are: load a state by copying
    into them.
    bind() names the gradients and the 16-bit parameters that step() reads and
    writes; without a param_dtype the fp32 master is all there is.  With
    statistics=False a step neither clips nor looks for an overflow.

    On one of several ranks the norm, the clip and the skip cover all of them:
    take the statistics first (zero_multi_unscale_norm on plan and state),
    exchange state.field("sumsq") and state.field("overflow"), put the others'
    into state.field("remote_sumsq") and state.field("remote_overflow"), and
    step with zero_multi_adamw_step on the arenas."""

    def __init__(self, masters, hp, state_bits=32, loss_scale=65536.0, dynamic=False, window=1000,
                 min_scale=1.0, lr_mult=None, decay_mult=None, statistics=True, seed=0,
                 grad_dtype=torch.bfloat16, param_dtype=torch.bfloat16):
        masters = list(masters)
        if not masters:
            raise ValueError("need at least one master tensor")
        for k, t in enumerate(masters):
            _dev(t, "masters[%d]" % k, ("float32",))
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 32 or 8")
        if not statistics and hp.get("max_grad_norm", 0.0) > 0.0:
            raise ValueError("clipping needs the statistics: max_grad_norm must be 0 without them")
        dev = masters[0].device
        n = [t.numel() for t in masters]
        self.plan = MultiPlan(n, grad_dtype, param_dtype, state_bits, device=dev)
        rows = [-(-x // ZERO_ROW) for x in n]
        self.first_row = [0] + list(itertools.accumulate(rows))[:-1]
        size = self.plan.rows * ZERO_ROW
        kinds = (torch.float8_e4m3fn, torch.float8_e5m2) if state_bits == 8 else (torch.float32,) * 2
        # rows without padding are filled by the copy below
        arenas = [(torch.zeros if any(x % ZERO_ROW for x in n) else torch.empty)(size, device=dev)]
        arenas += [torch.zeros(size * k.itemsize, dtype=torch.uint8, device=dev).view(k) for k in kinds]
        for _ in range(2):
            arenas.append(torch.zeros(self.plan.rows, device=dev) if state_bits == 8 else None)
        self._arenas = tuple(arenas)
        if size:
            # detached: a model's own parameters would make the arena part of a graph
            torch._foreach_copy_(self.views(self.master), [t.detach().view(-1) for t in masters])
        self.hp = dict(hp)
        self.statistics, self.seed = bool(statistics), int(seed)
        self.lr_mult, self.decay_mult = lr_mult, decay_mult
        self._state = StepState(loss_scale, dynamic, window, min_scale, device=dev)
        # the library call's arguments, of which only hp, seed and flags change
        self._args = zero_multi_step_args_t(
            C.addressof(self.plan._plan), self.plan._image_ptr,
            *[None if t is None else t.data_ptr() for t in arenas], self._state.ptr())
        self._ref = C.byref(self._args)
        self._args_of = None

    master = property(lambda self: self._arenas[0])
    exp_avg = property(lambda self: self._arenas[1])
    exp_avg_sq = property(lambda self: self._arenas[2])
    exp_avg_scale = property(lambda self: self._arenas[3])
    exp_avg_sq_scale = property(lambda self: self._arenas[4])
    state = property(lambda self: self._state)

    def views(self, arena):
        """The tensors inside an arena (flat views, without the rows' padding)."""
        return [arena[r * ZERO_ROW:r * ZERO_ROW + n]
                for r, n in zip(self.first_row, self.plan.numels)]

    def bind(self, grads, params=None):
        """Name the gradients and the 16-bit parameters; again whenever one of
        them is another tensor than before (see MultiPlan.bind)."""
        self.plan.bind(grads, params, self.lr_mult, self.decay_mult)

    def _refresh(self):
        """The arguments that the attributes hp, seed and statistics set."""
        if not self.statistics and self.hp.get("max_grad_norm", 0.0) > 0.0:
            raise ValueError("clipping needs the statistics: max_grad_norm must be 0 without them")
        self._args.hp = zero_adamw_hparams_t(**self.hp)
        self._args.seed = self.seed & 0xffffffff
        self._args.flags = ZERO_STEP_FINALIZE | (ZERO_MULTI_STATISTICS if self.statistics else 0)
        self._args_of = (dict(self.hp), self.seed, self.statistics)

    def step(self, stream=None):
        """Statistics over the bound gradients, then the step (one library call,
        as zero_multi_adamw_step with its arguments prepared).  On a stream
        other than the tensors' own, the caller orders the two, and keeps the
        optimizer until the step is done."""
        if not self.plan._bound:
            self.plan._require_bound()
        if self._args_of != (self.hp, self.seed, self.statistics):
            self._refresh()
        rc = _lib.zero_multi_adamw_step_args(
            self._ref, _current_raw_stream() if stream is None else _stream(stream))
        if rc:
            _check(rc)
