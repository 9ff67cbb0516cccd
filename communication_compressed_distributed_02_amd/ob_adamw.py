"""Python binding of the ob_adamw interface (argument marshalling only):
AdamW's step over many tensors with states in 32 bits or in 8, and the global
gradient norm.

Functions carry the names of include/ob_adamw.h and raise ObAdamError on a
status other than OB_OK.  Every computation runs in the library's HIP
kernels; PyTorch only provides device memory and the stream.
"""
import ctypes

import torch

from .ob_adam import _check, _lib, OnStream

OB_ADAMW_F32, OB_ADAMW_BF16 = 0, 1
OB_ADAMW_MAX_GROUPS = 32
(OB_ADAMW_M, OB_ADAMW_V, OB_ADAMW_MASTER, OB_ADAMW_M_EXP, OB_ADAMW_V_EXP) = range(5)

EXPORTED = ("ob_adamw_layout", "ob_adamw_init", "ob_adamw_attach", "ob_adamw_grad_norm",
            "ob_adamw_step", "ob_adamw_get_state", "ob_adamw_set_state", "ob_adamw_state",
            "ob_adamw_set_steps", "ob_adamw_get_steps", "ob_adamw_check_guards",
            "ob_adamw_set_stream", "ob_adamw_destroy")

FIELDS = {"m": OB_ADAMW_M, "v": OB_ADAMW_V, "master": OB_ADAMW_MASTER, "m_exp": OB_ADAMW_M_EXP,
          "v_exp": OB_ADAMW_V_EXP}
# the caller's current stream as a number: a tenth of the time of comparing
# Stream objects, which a step of a few microseconds notices
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_TYPES = {torch.float32: OB_ADAMW_F32, torch.bfloat16: OB_ADAMW_BF16}


class ob_adamw_config(ctypes.Structure):
    _fields_ = [("n_tensors", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("state_bits", ctypes.c_int32), ("master", ctypes.c_int32),
                ("stochastic", ctypes.c_int32), ("beta1", ctypes.c_float),
                ("beta2", ctypes.c_float), ("eps", ctypes.c_float), ("seed", ctypes.c_uint64)]


class ob_adamw_step_args(ctypes.Structure):
    _fields_ = [("lr", ctypes.POINTER(ctypes.c_float)),
                ("weight_decay", ctypes.POINTER(ctypes.c_float)),
                ("lr_device", ctypes.c_void_p), ("grad_scale", ctypes.c_float),
                ("max_norm", ctypes.c_float), ("skip_nonfinite", ctypes.c_int32),
                ("sumsq", ctypes.c_void_p), ("norm", ctypes.c_void_p)]


def _declare(L):
    P, I32, I64, U64, F = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                           ctypes.c_float)
    cfg, i64s, i32s = (ctypes.POINTER(ob_adamw_config), ctypes.POINTER(I64), ctypes.POINTER(I32))
    ptrs = ctypes.POINTER(P)
    sig = {
        "ob_adamw_layout": [cfg, i64s, i64s, i64s, ctypes.POINTER(U64)],
        "ob_adamw_init": [cfg, i64s, i32s, P, U64, ptrs, P, ptrs],
        "ob_adamw_attach": [cfg, i64s, i32s, P, U64, P, ptrs],
        "ob_adamw_grad_norm": [P, ptrs, F, P, P],
        "ob_adamw_step": [P, ptrs, ptrs, ctypes.POINTER(ob_adamw_step_args)],
        "ob_adamw_get_state": [P, I32, I64, I64, I32, P],
        "ob_adamw_set_state": [P, I32, I64, I64, P],
        "ob_adamw_state": [P, I32, ptrs, ctypes.POINTER(U64)],
        "ob_adamw_set_steps": [P, I64],
        "ob_adamw_get_steps": [P, i64s, i64s],
        "ob_adamw_check_guards": [P, i32s],
        "ob_adamw_set_stream": [P, P],
        "ob_adamw_destroy": [P],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int


_declare(_lib)


def make_config(n_tensors, n_groups=1, param_dtype=OB_ADAMW_F32, grad_dtype=OB_ADAMW_F32,
                state_bits=32, master=False, stochastic=False, beta1=0.9, beta2=0.999, eps=1e-8,
                seed=0):
    return ob_adamw_config(n_tensors, n_groups, param_dtype, grad_dtype, state_bits, int(master),
                           int(stochastic), beta1, beta2, eps, seed)


def _i64s(values):
    return (ctypes.c_int64 * max(1, len(values)))(*values)


def _numels(cfg, numels):
    if len(numels) != cfg.n_tensors:
        raise ValueError("%d element counts given for %d tensors" % (len(numels), cfg.n_tensors))
    return _i64s(numels)


def ob_adamw_layout(cfg, numels):
    """(first state element of every tensor, elements of a state array,
    workspace bytes)."""
    offsets = _i64s([0] * len(numels))
    length, total = ctypes.c_int64(0), ctypes.c_uint64(0)
    _check(_lib.ob_adamw_layout(ctypes.byref(cfg), _numels(cfg, numels), offsets,
                                ctypes.byref(length), ctypes.byref(total)), "ob_adamw_layout")
    return list(offsets)[:len(numels)], length.value, total.value


def _groups(cfg, groups):
    if groups is None:
        return None
    if len(groups) != cfg.n_tensors:
        raise ValueError("%d groups given for %d tensors" % (len(groups), cfg.n_tensors))
    return (ctypes.c_int32 * len(groups))(*groups)


def ob_adamw_init(cfg, numels, groups, workspace_ptr, ws_bytes, param_ptrs, stream_ptr):
    h = ctypes.c_void_p(0)
    _check(_lib.ob_adamw_init(ctypes.byref(cfg), _numels(cfg, numels), _groups(cfg, groups),
                              workspace_ptr, ws_bytes, param_ptrs, stream_ptr, ctypes.byref(h)),
           "ob_adamw_init")
    return h.value


def ob_adamw_attach(cfg, numels, groups, workspace_ptr, ws_bytes, stream_ptr):
    h = ctypes.c_void_p(0)
    _check(_lib.ob_adamw_attach(ctypes.byref(cfg), _numels(cfg, numels), _groups(cfg, groups),
                                workspace_ptr, ws_bytes, stream_ptr, ctypes.byref(h)),
           "ob_adamw_attach")
    return h.value


def ob_adamw_grad_norm(h, grad_ptrs, grad_scale, sumsq_ptr, norm_ptr):
    _check(_lib.ob_adamw_grad_norm(h, grad_ptrs, grad_scale, sumsq_ptr, norm_ptr),
           "ob_adamw_grad_norm")


def ob_adamw_step(h, param_ptrs, grad_ptrs, args):
    _check(_lib.ob_adamw_step(h, param_ptrs, grad_ptrs, args), "ob_adamw_step")


def ob_adamw_get_state(h, field, offset, count, dtype, dst_ptr):
    _check(_lib.ob_adamw_get_state(h, field, offset, count, dtype, dst_ptr), "ob_adamw_get_state")


def ob_adamw_set_state(h, field, offset, count, src_ptr):
    _check(_lib.ob_adamw_set_state(h, field, offset, count, src_ptr), "ob_adamw_set_state")


def ob_adamw_state(h, field):
    """(device address, bytes) of a field as it is stored."""
    p, n = ctypes.c_void_p(0), ctypes.c_uint64(0)
    _check(_lib.ob_adamw_state(h, field, ctypes.byref(p), ctypes.byref(n)), "ob_adamw_state")
    return p.value, n.value


def ob_adamw_set_steps(h, steps):
    _check(_lib.ob_adamw_set_steps(h, steps), "ob_adamw_set_steps")


def ob_adamw_get_steps(h):
    a, b = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(_lib.ob_adamw_get_steps(h, ctypes.byref(a), ctypes.byref(b)), "ob_adamw_get_steps")
    return a.value, b.value


def ob_adamw_check_guards(h):
    """-1 if every workspace guard is intact, else the first changed one."""
    bad = ctypes.c_int32(0)
    _check(_lib.ob_adamw_check_guards(h, ctypes.byref(bad)), "ob_adamw_check_guards")
    return bad.value


def ob_adamw_set_stream(h, stream_ptr):
    _check(_lib.ob_adamw_set_stream(h, stream_ptr), "ob_adamw_set_stream")


def ob_adamw_destroy(h):
    _check(_lib.ob_adamw_destroy(h), "ob_adamw_destroy")


class TensorBatch:
    """One step's gradients and the parameters they belong to, checked and
    marshalled once (bind); the calls take it in place of the list and skip the
    per-call checks.  It holds the tensors, whose contents may change."""
    __slots__ = ("plan", "grads", "params", "tensors", "grad_ptrs", "param_ptrs")

    def __init__(self, plan, grads, grad_ptrs, params, param_ptrs):
        self.plan, self.grads, self.params = plan, grads, params
        self.tensors = tuple(t for t in (*grads, *params) if t is not None)
        self.grad_ptrs, self.param_ptrs = grad_ptrs, param_ptrs

    def __len__(self):
        return len(self.grads)


class _Plan(OnStream):
    """A handle over a list of tensors' sizes and its workspace."""

    def __init__(self, numels, groups, cfg, grad_dtype, device, stream, checkpoint=None,
                 params=None):
        self.cfg, self.numels, self.grad_dtype = cfg, list(numels), grad_dtype
        self.groups = None if groups is None else [int(g) for g in groups]
        _groups(cfg, self.groups)
        self.h = None
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("tensors on %s: a GPU is needed" % self.device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._not_capturing()
        self.offsets, self.length, self.ws_bytes = ob_adamw_layout(cfg, self.numels)
        with torch.cuda.device(self.device):
            self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
            self._stream_ptr = self.stream.cuda_stream
            if checkpoint is not None:
                self._check_bytes(checkpoint)
            # what results are made like: a third less time than naming a type and device
            self._like_norm = torch.empty((), dtype=torch.float32, device=self.device)
            self._like_sumsq = torch.empty((), dtype=torch.float64, device=self.device)
            self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
            self._order_after_caller(self.workspace)
            if checkpoint is not None:
                self.h = self._adopt(checkpoint)
            else:
                self.h = ob_adamw_init(cfg, self.numels, self.groups, self.workspace.data_ptr(),
                                       self.ws_bytes, params, self.stream.cuda_stream)

    def _check_bytes(self, checkpoint):
        if checkpoint.dtype != torch.uint8:
            raise ValueError("a checkpoint is a uint8 tensor, not " + str(checkpoint.dtype))
        if checkpoint.numel() != self.ws_bytes:
            raise ValueError("checkpoint of %d bytes, workspace needs %d"
                             % (checkpoint.numel(), self.ws_bytes))

    def _adopt(self, checkpoint):
        """A handle over the workspace with the checkpoint's bytes in it, made on
        the plan's stream, which is waited for."""
        with torch.cuda.stream(self.stream):
            self.workspace.copy_(checkpoint)
        return ob_adamw_attach(self.cfg, self.numels, self.groups, self.workspace.data_ptr(),
                               self.ws_bytes, self.stream.cuda_stream)

    def _call(self, lists, fn, *args):
        """fn(*args) with this plan's device current, ordered with the
        caller's stream; lists: of the tensors it touches.  On a stream under
        capture the call is recorded there (the plan's own stream may be the
        default one, which cannot take part in a capture)."""
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                self._call(lists, fn, *args)
            return
        current = _current_stream(self.device.index)
        if current == self._stream_ptr:
            fn(*args)
        elif torch.cuda.is_current_stream_capturing():
            ob_adamw_set_stream(self.h, current)
            try:
                fn(*args)
            finally:
                ob_adamw_set_stream(self.h, self._stream_ptr)
        else:
            self._ordered([t for some in lists for t in some], fn, *args)

    def _ptrs(self, tensors, dtype, what, may_lack):
        if len(tensors) != len(self.numels):
            raise ValueError("%d %s given, %d expected" % (len(tensors), what, len(self.numels)))
        ptrs = (ctypes.c_void_p * len(tensors))()
        for i, (t, n) in enumerate(zip(tensors, self.numels)):
            if t is None:
                if not may_lack:
                    raise ValueError("%s %d is missing" % (what, i))
                continue
            if (t.dtype != dtype or t.numel() != n or t.device != self.device
                    or not t.is_contiguous()):
                raise ValueError("%s %d must be a contiguous %s tensor of %d elements on %s"
                                 % (what, i, dtype, n, self.device))
            ptrs[i] = t.data_ptr()
        return ptrs

    def grad_norm(self, grads, grad_scale=1.0):
        """(norm as a float32 scalar, sum of squares as a float64 scalar) of
        the gradients (None: no gradient), on the device."""
        b = grads
        if not isinstance(b, TensorBatch):
            grads = tuple(grads)
            b = TensorBatch(self, grads, self._ptrs(grads, self.grad_dtype, "gradients", True), (),
                            None)
        if b.plan is not self:
            raise ValueError("a batch bound by another plan")
        norm, sumsq = torch.empty_like(self._like_norm), torch.empty_like(self._like_sumsq)
        self._call((b.tensors, (norm, sumsq)), ob_adamw_grad_norm, self.h, b.grad_ptrs, grad_scale,
                   sumsq.data_ptr(), norm.data_ptr())
        return norm, sumsq

    @staticmethod
    def _not_capturing():
        """Raises where the current stream is under capture, before anything is
        enqueued there or waited for, so that the capture goes on."""
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("this call waits for the GPU: not while a graph is captured")

    def _wait(self, fn):
        """fn(handle), a call that waits for the plan's stream, and before it for
        the caller's, where graphs of the plan's calls may have been replayed."""
        self._not_capturing()
        torch.cuda.current_stream(self.device).synchronize()
        with torch.cuda.device(self.device):
            return fn(self.h)

    def check_guards(self):
        """-1 if no kernel wrote past a workspace buffer (synchronizes)."""
        return self._wait(ob_adamw_check_guards)

    def close(self):
        if self.h:
            ob_adamw_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class GradNorm(_Plan):
    """The global norm of gradients of the sizes, type and device of
    `tensors` (gradients, or parameters with `grad_dtype`)."""

    def __init__(self, tensors, grad_dtype=None, stream=None):
        tensors = list(tensors)
        if not tensors:
            raise ValueError("no tensors")
        dt = tensors[0].dtype if grad_dtype is None else grad_dtype
        if dt not in _TYPES:
            raise ValueError("gradients are float32 or bfloat16")
        cfg = make_config(len(tensors), grad_dtype=_TYPES[dt], state_bits=0)
        super().__init__([t.numel() for t in tensors], None, cfg, dt, tensors[0].device, stream)

    def bind(self, grads):
        """A TensorBatch of the gradients (checked here once)."""
        grads = tuple(grads)
        return TensorBatch(self, grads, self._ptrs(grads, self.grad_dtype, "gradients", True), (),
                           None)


class AdamW(_Plan):
    """AdamW over `params` (contiguous float32 or bfloat16 tensors of one type
    on one device), which the steps update where they lie.

    groups: each tensor's hyperparameter group (default all 0) of `n_groups`
    (default: as many as are named; at most OB_ADAMW_MAX_GROUPS).  grad_dtype:
    the gradients' type (default the parameters').  state_bits: 32 or 8.
    master: keep float32 copies of bfloat16 parameters, taken now: the steps go
    on from the copies (`views()`, `set`), not from parameters that are written
    between them.  stochastic: round bfloat16 parameters without copies
    stochastically.  seed: of the random
    bits.  steps: steps already taken.  checkpoint: the workspace bytes of
    checkpoint() of a plan with the same configuration and sizes."""

    def __init__(self, params, groups=None, n_groups=None, grad_dtype=None, state_bits=32,
                 master=False, stochastic=False, betas=(0.9, 0.999), eps=1e-8, seed=0, steps=0,
                 stream=None, checkpoint=None):
        params = tuple(params)
        if not params:
            raise ValueError("no parameters")
        dt = params[0].dtype
        gdt = dt if grad_dtype is None else grad_dtype
        if dt not in _TYPES or gdt not in _TYPES:
            raise ValueError("parameters and gradients are float32 or bfloat16")
        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        self.param_dtype = dt
        groups = None if groups is None else tuple(groups)
        self.n_groups = n_groups or (1 if groups is None else max(groups) + 1)
        cfg = make_config(len(params), self.n_groups, _TYPES[dt], _TYPES[gdt], state_bits, master,
                          stochastic, betas[0], betas[1], eps, seed)
        # checked as _ptrs does, before the workspace exists
        self.device, self.numels = params[0].device, [p.numel() for p in params]
        ptrs = self._ptrs(params, dt, "parameters", False)
        self.params = params
        super().__init__(self.numels, groups, cfg, gdt, self.device, stream, checkpoint,
                         ptrs if master else None)
        if checkpoint is None and steps:
            self.set_steps(steps)
        self._args = ob_adamw_step_args()
        self._lr = (ctypes.c_float * self.n_groups)()
        self._wd = (ctypes.c_float * self.n_groups)()
        self._args.lr = ctypes.cast(self._lr, ctypes.POINTER(ctypes.c_float))
        self._args.weight_decay = ctypes.cast(self._wd, ctypes.POINTER(ctypes.c_float))
        self._args_ref = ctypes.byref(self._args)

    def bind(self, grads, params=None):
        """A TensorBatch of one step's gradients (None: the tensor is left as
        it is) and the parameters as they lie now (checked here once)."""
        grads = tuple(grads)
        params = self.params if params is None else tuple(params)
        return TensorBatch(self, grads, self._ptrs(grads, self.grad_dtype, "gradients", True),
                           params, self._ptrs(params, self.param_dtype, "parameters", False))

    def _per_group(self, values, into, what):
        if not hasattr(values, "__len__"):
            for i in range(self.n_groups):
                into[i] = values
            return
        if len(values) != self.n_groups:
            raise ValueError("%d %s given for %d groups" % (len(values), what, self.n_groups))
        into[:] = values

    def step(self, grads, lr, weight_decay=0.0, max_norm=0.0, grad_scale=1.0,
             skip_nonfinite=False, sumsq=None):
        """One step.  grads: a list (None: left as it is) or a TensorBatch.
        lr, weight_decay: a number, or one per group; lr may be a float32
        device tensor of n_groups elements, read when the step runs.
        max_norm: clip by the global norm (0: no clipping).  sumsq: a float64
        device scalar to clip and skip by in place of these gradients' own.
        Returns the norm as a float32 device scalar where it clips or skips,
        else None."""
        b = grads if isinstance(grads, TensorBatch) else self.bind(grads)
        if b.plan is not self:
            raise ValueError("a batch bound by another plan")
        a, more = self._args, []
        if isinstance(lr, torch.Tensor):
            if (lr.dtype != torch.float32 or lr.numel() != self.n_groups
                    or lr.device != self.device or not lr.is_contiguous()):
                raise ValueError("lr must be a contiguous float32 tensor of %d elements on %s"
                                 % (self.n_groups, self.device))
            a.lr_device = lr.data_ptr()
            more.append(lr)
        else:
            a.lr_device = None
            self._per_group(lr, self._lr, "learning rates")
        self._per_group(weight_decay, self._wd, "weight decays")
        a.grad_scale, a.max_norm, a.skip_nonfinite = grad_scale, max_norm, bool(skip_nonfinite)
        if sumsq is not None:
            if (sumsq.dtype != torch.float64 or sumsq.numel() != 1
                    or sumsq.device != self.device):
                raise ValueError("sumsq must be a float64 scalar on %s" % self.device)
            a.sumsq = sumsq.data_ptr()
            more.append(sumsq)
        else:
            a.sumsq = None
        norm = None
        if max_norm or skip_nonfinite:
            norm = torch.empty_like(self._like_norm)
            a.norm = norm.data_ptr()
            more.append(norm)
        else:
            a.norm = None
        self._call((b.tensors, more), ob_adamw_step, self.h, b.param_ptrs, b.grad_ptrs, self._args_ref)
        return norm

    def views(self):
        """Tensors aliasing the state as it is stored (the state layout:
        tensor i from element offsets[i]): float32 m and v, or the e4m3 codes m
        and the codes v with one exponent byte per 256 elements, m_exp and
        v_exp; and the float32 master copies, if there are any."""
        names = ["m", "v"] + (["m_exp", "v_exp"] if self.cfg.state_bits == 8 else []) + (
            ["master"] if self.cfg.master else [])
        base, out = self.workspace.data_ptr(), {}
        for name in names:
            p, n = ob_adamw_state(self.h, FIELDS[name])
            out[name] = self.workspace[p - base:p - base + n]
            if name == "master" or (name in ("m", "v") and self.cfg.state_bits == 32):
                out[name] = out[name].view(torch.float32)
            elif name == "m":
                out[name] = out[name].view(torch.float8_e4m3fn)
        return out

    def get(self, name, tensor=None, dtype=torch.float32):
        """Values of "m", "v" or "master" as a new tensor: of one tensor, or
        the whole state array in the state layout."""
        if dtype not in _TYPES:
            raise ValueError("state is read as float32 or bfloat16")
        offset, count = (0, self.length) if tensor is None else (self.offsets[tensor],
                                                                 self.numels[tensor])
        out = torch.empty(count, dtype=dtype, device=self.device)
        self._call(((out,),), ob_adamw_get_state, self.h, FIELDS[name], offset, count, _TYPES[dtype],
                   out.data_ptr() if count else None)
        return out

    def set(self, name, src, tensor):
        """Overwrite "m", "v" or "master" of one tensor from float32 values
        (8-bit states are encoded, rounded to nearest)."""
        n = self.numels[tensor]
        if src.dtype != torch.float32 or src.numel() != n or src.device != self.device:
            raise ValueError("source must be a float32 tensor of %d elements on %s"
                             % (n, self.device))
        rows = -(-n // 1024) * 1024
        whole = torch.zeros(rows, dtype=torch.float32, device=self.device)
        whole[:n].copy_(src.reshape(-1))
        self._call(((whole,),), ob_adamw_set_state, self.h, FIELDS[name], self.offsets[tensor], rows,
                   whole.data_ptr() if n else None)

    def set_steps(self, steps):
        self._call((), ob_adamw_set_steps, self.h, steps)

    @property
    def steps(self):
        """(steps taken, steps skipped), replays among them (synchronizes)."""
        return self._wait(ob_adamw_get_steps)

    def load(self, checkpoint):
        """Go on from the workspace bytes of checkpoint() of a plan with the
        same configuration and sizes.  They are copied to where the workspace
        lies, so graphs captured from this plan go on from them too.
        (Synchronizes.)"""
        self._check_bytes(checkpoint)
        self._not_capturing()
        with torch.cuda.device(self.device):
            self._order_after_caller()
            h = self._adopt(checkpoint)
        self.close()
        self.h = h

    def checkpoint(self, device="cpu"):
        """A copy of the workspace bytes: the whole optimizer state.  Taken on
        the plan's stream, between what the caller's holds so far and the calls
        that follow, from whichever stream they come."""
        self._not_capturing()
        with torch.cuda.device(self.device):
            self._order_after_caller()
            with torch.cuda.stream(self.stream):
                copy = self.workspace.to(device, copy=True)
            if self._separate():
                current = torch.cuda.current_stream(self.device)
                current.wait_stream(self.stream)
                if copy.device == self.device:
                    copy.record_stream(current)
        return copy
