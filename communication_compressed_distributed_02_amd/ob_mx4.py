"""Python binding of the ob_mx4 interface: matrices in microscaled 4-bit
floating point (blocks of 32 elements that share a power of two), their
products, and a linear layer made of them.

    q = quantize(x)                     # x: float32 or bfloat16, blocks along its last dimension
    rows, cols = quantize_both(x)       # x and its transpose, from one read
    q.dequantize()                      # back to float32 or bfloat16
    msg = quantize(g, seed=s, residual=e)      # a worker's message, with error feedback
    mean = average(messages)            # of several workers
    y = matmul(a, b)                    # a b^T on the matrix cores; a may be a plain tensor
    y = linear(x, weight, seed=s)       # differentiable; all three products in 4 bits

Gradients pass through linear alone: while they are recorded, an input of matmul
and tensors that are written may not want one.  An MX4 holds values only.

Functions work on the current stream of their tensors' device, as torch's own
do, and may be captured in a graph.  They raise ValueError on tensors that do
not fit and ObAdamError on a status other than OB_OK.  Every computation runs
in the library's HIP kernels; there is no fallback.
"""
import ctypes
import math
import weakref

import torch

from .ob_adam import _check, _lib

OB_MX4_F32, OB_MX4_BF16 = 0, 1
OB_MX4_MAX_MESSAGES = 64

EXPORTED = ("ob_mx4_layout", "ob_mx4_quantize", "ob_mx4_average", "ob_mx4_matmul_workspace",
            "ob_mx4_matmul")

_TYPES = {torch.float32: OB_MX4_F32, torch.bfloat16: OB_MX4_BF16}
# the caller's current stream as a number (see ob_adamw)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class ob_mx4_quantize_args(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("stochastic", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("stride", ctypes.c_int64),
                ("seed", ctypes.c_uint64), ("seed_device", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("codes_t", ctypes.c_void_p),
                ("scales_t", ctypes.c_void_p)]


class ob_mx4_matmul_args(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("a_codes", ctypes.c_void_p), ("a_scales", ctypes.c_void_p),
                ("a", ctypes.c_void_p), ("a_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("a_stride", ctypes.c_int64), ("b_codes", ctypes.c_void_p),
                ("b_scales", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_int64), ("accumulate", ctypes.c_int32),
                ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_uint64)]


def _declare(L):
    P, I32, I64, U64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
    ptrs, i64s = ctypes.POINTER(P), ctypes.POINTER(I64)
    product = ctypes.POINTER(ob_mx4_matmul_args)
    sig = {
        "ob_mx4_layout": [I64, I64, i64s, i64s],
        "ob_mx4_quantize": [ctypes.POINTER(ob_mx4_quantize_args), P],
        "ob_mx4_average": [ptrs, ptrs, I32, I64, I64, I32, P, I64, P],
        "ob_mx4_matmul_workspace": [product, ctypes.POINTER(U64)],
        "ob_mx4_matmul": [product, P],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int


_declare(_lib)


def ob_mx4_layout(rows, cols):
    """Bytes of (a row of codes, a row of scales)."""
    codes, scales = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(_lib.ob_mx4_layout(rows, cols, ctypes.byref(codes), ctypes.byref(scales)),
           "ob_mx4_layout")
    return codes.value, scales.value


def ob_mx4_quantize(args, stream_ptr):
    _check(_lib.ob_mx4_quantize(ctypes.byref(args), stream_ptr), "ob_mx4_quantize")


_POINTERS = [ctypes.c_void_p * n for n in range(OB_MX4_MAX_MESSAGES + 2)]


def ob_mx4_average(code_ptrs, scale_ptrs, rows, cols, dtype, out_ptr, stride, stream_ptr):
    n = len(code_ptrs)
    array = _POINTERS[n] if n < len(_POINTERS) else ctypes.c_void_p * n
    _check(_lib.ob_mx4_average(array(*code_ptrs), array(*scale_ptrs), n, rows, cols, dtype, out_ptr,
                               stride, stream_ptr), "ob_mx4_average")


def ob_mx4_matmul_workspace(args):
    out = ctypes.c_uint64(0)
    _check(_lib.ob_mx4_matmul_workspace(ctypes.byref(args), ctypes.byref(out)),
           "ob_mx4_matmul_workspace")
    return out.value


def ob_mx4_matmul(args, stream_ptr):
    _check(_lib.ob_mx4_matmul(ctypes.byref(args), stream_ptr), "ob_mx4_matmul")


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(device, fn, *args):
    """fn(*args, stream) with `device` current, on its current stream."""
    index = device.index  # None off the GPU
    if index is None or _current_device() != index:
        if device.type != "cuda":
            raise ValueError("a quantised matrix on %s: a GPU is needed" % device)
        with torch.cuda.device(device):
            fn(*args, _current_stream(index))
    else:
        fn(*args, _current_stream(index))


def _widths(cols):
    """Bytes of a row of codes and of a row of scales (ob_mx4_layout, of sizes that
    a tensor has already)."""
    return (cols + 127) // 128 * 64, (cols + 511) // 512 * 16


def _need_gpu(t, what):
    if t.device.type != "cuda":
        raise ValueError("%s on %s: a GPU is needed" % (what, t.device))


class MX4:
    """A quantised matrix: `codes` and `scales` as uint8 matrices in the layout
    of include/ob_mx4.h, and its number of columns.  The tensors' memory is taken
    as it is, not copied.  It may be copied, deep-copied, pickled and saved (to
    torch's safe loader MX4 has to be named); calls take one on a GPU."""
    __slots__ = ("rows", "cols", "device", "code_ptr", "scale_ptr", "_held")

    def __init__(self, codes, scales, cols):
        for t, what in ((codes, "codes"), (scales, "scales")):
            if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_contiguous():
                raise ValueError("%s must be a contiguous uint8 matrix" % what)
            _need_gpu(t, what)
            if t.data_ptr() % 16:
                raise ValueError("%s must be aligned to 16 bytes" % what)
        width = ob_mx4_layout(codes.shape[0], cols)
        if (codes.shape[1], scales.shape[1]) != width or scales.shape[0] != codes.shape[0]:
            raise ValueError("codes %s and scales %s are not those of %d columns"
                             % (tuple(codes.shape), tuple(scales.shape), cols))
        if codes.device != scales.device:
            raise ValueError("codes on %s, scales on %s" % (codes.device, scales.device))
        # aliases, which stay there should the caller's be given other memory
        self._place(codes.shape[0], cols, (codes.detach(), scales.detach()))

    @classmethod
    def empty(cls, rows, cols, device):
        """One with undefined contents."""
        ob_mx4_layout(rows, cols)
        some = torch.empty(0, dtype=torch.uint8, device=device)
        _need_gpu(some, "a quantised matrix")
        return cls._like(some, rows, cols)

    @classmethod
    def _like(cls, x, rows, cols):
        """One with undefined contents where the tensor x lies: codes and scales
        in one allocation, made views of when they are asked for."""
        return cls._over(x.new_empty(rows * sum(_widths(cols)), dtype=torch.uint8), rows, cols)

    @classmethod
    def _over(cls, held, rows, cols):
        """One whose codes and then scales fill `held`."""
        q = object.__new__(cls)
        q._place(rows, cols, held)
        return q

    # What is copied or sent are the tensors alone: where they lie is read off the
    # ones that arrive.  (Read off at every call it costs 0.1 us a pointer and more:
    # an average of 4 small messages 9.1 us for 7.2.)
    def __getstate__(self):
        return self.rows, self.cols, self._held

    def __setstate__(self, state):
        self._place(*state)

    def _place(self, rows, cols, held):
        self.rows, self.cols, self._held = rows, cols, held
        if isinstance(held, tuple):
            self.device = held[0].device
            self.code_ptr, self.scale_ptr = held[0].data_ptr(), held[1].data_ptr()
        else:
            self.device, self.code_ptr = held.device, held.data_ptr()
            self.scale_ptr = self.code_ptr + rows * _widths(cols)[0]

    def _part(self, i):
        if isinstance(self._held, tuple):
            return self._held[i]
        width = _widths(self.cols)[i]
        begin = (self.scale_ptr if i else self.code_ptr) - self._held.data_ptr()
        return self._held[begin:begin + self.rows * width].view(self.rows, width)

    @property
    def codes(self):
        return self._part(0)

    @property
    def scales(self):
        return self._part(1)

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def nbytes(self):
        return self.rows * sum(_widths(self.cols))

    def dequantize(self, dtype=torch.float32, out=None):
        """Its values as float32 or bfloat16."""
        return average((self,), dtype, out)

    def __repr__(self):
        return "MX4(%d x %d on %s)" % (self.rows, self.cols, self.device)


def _matrix(x, what):
    """x as a matrix (dimensions in front of the last joined; a vector is one row)."""
    if x.dtype not in _TYPES:
        raise ValueError("%s must be float32 or bfloat16, not %s" % (what, x.dtype))
    _need_gpu(x, what)
    if x.dim() == 2:
        return x
    if x.dim() == 0:
        raise ValueError("%s must have a dimension" % what)
    try:
        return x.view(math.prod(x.shape[:-1]), x.shape[-1])
    except RuntimeError:
        raise ValueError("%s of shape %s and strides %s is no matrix: make it contiguous"
                         % (what, tuple(x.shape), x.stride())) from None


def _no_gradient(t, what):
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("no gradient passes through %s, which wants one: detach it, or use linear"
                         % what)


# (a half of the time of torch.autograd.graph.increment_version, which calls it)
_count_write = getattr(torch._C, "_increment_version", None) or torch.autograd.graph.increment_version


def _wrote(t):
    """Count a call's write to a tensor, or to a pair of them, as torch counts its own."""
    if isinstance(t, tuple):
        for part in t:
            _wrote(part)
    elif not t.is_inference():
        _count_write((t,))


def _by_rows(x):
    return x.stride(1) == 1 or x.shape[1] <= 1


def _row_stride(x):
    """Elements between rows (of a single row any will do)."""
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _target(out, rows, cols, x, what):
    if out is None:
        return MX4._like(x, rows, cols)
    if out.rows != rows or out.cols != cols or out.device != x.device:
        raise ValueError("%s must be %d x %d on %s, not %r" % (what, rows, cols, x.device, out))
    return out


def _quantize(x, seed, residual, rows, cols):
    """x by rows; rows: the MX4 of x or None, cols: that of its transpose or None."""
    m, n = x.shape
    device = x.device
    where = None
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1 or seed.device != device:
            raise ValueError("a seed is a number or an int64 scalar on %s" % device)
        where = seed.data_ptr()
    a = ob_mx4_quantize_args(
        x.data_ptr(), _TYPES[x.dtype], seed is not None, m, n, x.stride(0) if m > 1 else n,
        0 if seed is None or where is not None else seed & 0xFFFFFFFFFFFFFFFF, where,
        None if residual is None else residual.data_ptr(), None if rows is None else rows.code_ptr,
        None if rows is None else rows.scale_ptr, None if cols is None else cols.code_ptr,
        None if cols is None else cols.scale_ptr)
    _on(device, ob_mx4_quantize, a)


def quantize(x, seed=None, residual=None, out=None):
    """The MX4 of x (float32 or bfloat16), in blocks along its last dimension;
    dimensions in front of it are joined.  One dimension of the matrix has to be
    contiguous, either one.

    seed: round stochastically with these random bits (a number, or an int64
    device scalar that is read when the call runs); None rounds to nearest.  The bits
    go by the seed and the place in the matrix alone: every step, worker and tensor
    needs a seed of its own, or they round alike and their errors do not average out.
    residual: contiguous float32 of x's shape, added to x and replaced by what the
    rounding left (error feedback).  Where a value is not finite its block's message
    and residual are NaN, and so are those of later messages until the residual is
    cleared (residual.nan_to_num_(0.0)).  out: an MX4 to write to."""
    m = _matrix(x, "x")
    flip = not _by_rows(m)
    if flip and m.stride(0) != 1 and m.shape[0] > 1:
        raise ValueError("x has strides %s: one dimension must be contiguous" % (m.stride(),))
    if residual is not None:
        if (residual.dtype != torch.float32 or residual.shape != x.shape
                or residual.device != x.device or not residual.is_contiguous()):
            raise ValueError("the residual must be a contiguous float32 tensor of x's shape on %s"
                             % x.device)
        _no_gradient(residual, "the residual")
        if flip:
            raise ValueError("with a residual, x must be contiguous along its last dimension")
    given, out = out, _target(out, m.shape[0], m.shape[1], x, "out")
    if flip:
        _quantize(m.t(), seed, None, None, out)
    else:
        _quantize(m, seed, residual, out, None)
    if residual is not None:
        _wrote(residual)
    if given is not None:
        _wrote(given._held)
    return out


def quantize_both(x, seed=None, out=None):
    """(quantize(x), quantize(x.t())) of a matrix, from one read.  seed: as for
    quantize.  out: a pair to write to."""
    m = _matrix(x, "x")
    flip = not _by_rows(m)
    if flip and m.stride(0) != 1 and m.shape[0] > 1:
        raise ValueError("x has strides %s: one dimension must be contiguous" % (m.stride(),))
    rows, cols = (None, None) if out is None else out
    rows = _target(rows, m.shape[0], m.shape[1], x, "the first of out")
    cols = _target(cols, m.shape[1], m.shape[0], x, "the second of out")
    if flip:
        _quantize(m.t(), seed, None, cols, rows)
    else:
        _quantize(m, seed, None, rows, cols)
    if out is not None:
        _wrote(rows._held)
        _wrote(cols._held)
    return rows, cols


def _result(out, rows, cols, dtype, device):
    """The tensor that a call writes: `out` checked, or a new one."""
    if dtype not in _TYPES:
        raise ValueError("results are float32 or bfloat16, not %s" % dtype)
    if out is None:
        return torch.empty(rows, cols, dtype=dtype, device=device)
    if (tuple(out.shape) != (rows, cols) or out.dtype != dtype or out.device != device
            or not _by_rows(out) or (rows > 1 and out.stride(0) < cols)):
        raise ValueError("out must be %d x %d of %s on %s, rows contiguous and apart"
                         % (rows, cols, dtype, device))
    _no_gradient(out, "out")
    return out


def average(messages, dtype=torch.float32, out=None):
    """The mean of 1 to 64 MX4 of one shape, as float32 or bfloat16."""
    messages = tuple(messages)
    if not messages:
        raise ValueError("no messages")
    first = messages[0]
    for q in messages[1:]:
        if q.rows != first.rows or q.cols != first.cols or q.device != first.device:
            raise ValueError("messages differ: %r and %r" % (first, q))
    given, out = out, _result(out, first.rows, first.cols, dtype, first.device)
    _on(first.device, ob_mx4_average, [q.code_ptr for q in messages],
        [q.scale_ptr for q in messages], first.rows, first.cols, _TYPES[dtype],
        out.data_ptr(), _row_stride(out))
    if given is not None:
        _wrote(given)
    return out


_needs = {}


def _workspace(args, m, n, k, plain):
    """ob_mx4_matmul_workspace, which goes by these alone, of sizes asked for
    before."""
    key = m, n, k, plain
    need = _needs.get(key)
    if need is None:
        if len(_needs) >= 4096:
            _needs.clear()
        need = _needs[key] = ob_mx4_matmul_workspace(args)
    return need


def matmul(a, b, dtype=torch.bfloat16, out=None, accumulate=False):
    """a b^T: a is M x K, b N x K, the result M x N of float32 or bfloat16.

    b: an MX4.  a: an MX4, or a float32 or bfloat16 tensor, which is quantised
    to nearest on the way (its dimensions in front of the last are those of the
    result).  out: a matrix to write to; accumulate: add to it."""
    if isinstance(a, MX4):
        shape, rows, cols, device = None, a.rows, a.cols, a.device
        given = a.code_ptr, a.scale_ptr, None, 0
        stride = 0
    else:
        m = _matrix(a, "a")
        _no_gradient(a, "a")
        if not _by_rows(m):
            raise ValueError("a has strides %s: its last dimension must be contiguous"
                             % (m.stride(),))
        (rows, cols), device = m.shape, m.device
        shape = a.shape[:-1]
        given = None, None, m.data_ptr(), _TYPES[m.dtype]
        stride = m.stride(0) if rows > 1 else cols
    if cols != b.cols or device != b.device:
        raise ValueError("a of %d columns on %s, b %r" % (cols, device, b))
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    c = _result(out, rows, b.rows, dtype, device)
    _product(given, stride, rows, cols, b, c, dtype, accumulate)
    if out is not None:
        _wrote(out)
    if shape is not None and len(shape) != 1 and out is None:
        return c.view(*shape, b.rows)
    return c


def _product(given, stride, rows, cols, b, c, dtype, accumulate=False):
    """c = a b^T, or added to it; given: a's codes, scales, plain elements and
    their type."""
    args = ob_mx4_matmul_args(rows, b.rows, cols, *given, _TYPES[dtype], stride, b.code_ptr,
                              b.scale_ptr, c.data_ptr(), c.stride(0) if rows > 1 else b.rows,
                              accumulate, None, 0)
    need = _workspace(args, rows, b.rows, cols, given[0] is None)
    if need:
        # freed to torch's allocator on return: later work of this stream may have it then
        scratch = c.new_empty(need, dtype=torch.uint8)
        args.workspace, args.ws_bytes = scratch.data_ptr(), need
    _on(b.device, ob_mx4_matmul, args)


class Weight:
    """A weight's 4-bit copies: `rows` (N x K) for the forward product, `cols` (K x N)
    for the gradient of the input."""
    # _of, _seen: the tensor they were written from, and where it lay and its count of
    # writes then.  Not copied or sent along: another tensor counts otherwise.
    __slots__ = ("rows", "cols", "version", "_of", "_seen")

    def __init__(self, weight):
        self.rows, self.cols = quantize_both(weight.detach())
        self.version = 0
        self._of, self._seen = weakref.ref(weight), _writes(weight)

    def refresh(self, weight):
        """Written again, where they lie, from the weight as it is now."""
        quantize_both(weight.detach(), out=(self.rows, self.cols))
        self.version += 1
        self._of, self._seen = weakref.ref(weight), _writes(weight)
        return self

    def __getstate__(self):
        return self.rows, self.cols, self.version

    def __setstate__(self, state):
        self.rows, self.cols, self.version = state
        self._of = self._seen = None

    def behind(self, weight):
        """Whether `weight` is the tensor that they were written from and was written
        or moved since, as far as torch counts: writes through .data and by replays of
        a graph are not.  Of a Weight that was copied or loaded nothing is known."""
        return (self._of is not None and self._of() is weight
                and self._seen != _writes(weight))


def _writes(t):
    """Where a tensor lies and torch's count of the writes to it."""
    return t.data_ptr(), None if t.is_inference() else t._version


def _unit(x):
    """x as a matrix that quantize_both takes (a copy where it has to be)."""
    m = x if x.dim() == 2 else x.reshape(math.prod(x.shape[:-1]), x.shape[-1])
    return m if _by_rows(m) or m.stride(0) == 1 else m.contiguous()


def _of_mx4(a, b, like, dtype, shape=None):
    """a b^T of two MX4 that fit, as a new tensor where `like` lies."""
    c = like.new_empty((a.rows, b.rows), dtype=dtype)
    _product((a.code_ptr, a.scale_ptr, None, 0), 0, a.rows, a.cols, b, c, dtype)
    return c if shape is None or len(shape) == 2 else c.view(shape)


def _forward(x, m, a, w):
    """The layer's output: of a, x quantised, or where that is None of m, x as a
    matrix by rows, which is quantised on the way."""
    shape = (*x.shape[:-1], w.rows)
    if a is None:
        return matmul(m, w, x.dtype).view(shape)
    return _of_mx4(a, w, m, x.dtype, shape)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, quantized, seed):
        need_x, need_w = ctx.needs_input_grad[:2]
        m = _unit(x)
        a = x_cols = w_cols = None
        if quantized is not None:
            w, ctx.version = quantized.rows, quantized.version
        elif need_x:
            w, w_cols = quantize_both(weight)
        else:
            w = quantize(weight)
        if need_w:
            a, x_cols = quantize_both(m)
        elif not _by_rows(m):
            a = quantize(m)
        ctx.quantized, ctx.seed, ctx.x_shape, ctx.x_dtype = quantized, seed, x.shape, x.dtype
        ctx.w_shape, ctx.w_dtype = weight.shape, weight.dtype
        # as tensors of the graph's, so that it frees them behind the backward pass
        # and hooks on saved tensors (checkpointing) have them
        ctx.save_for_backward(None if x_cols is None else x_cols._held,
                              None if w_cols is None else w_cols._held)
        return _forward(x, m, a, w)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        need_x, need_w = ctx.needs_input_grad[:2]
        x_held, w_held = ctx.saved_tensors
        n, k = ctx.w_shape
        # dx alone reads them.  (Replays of a captured refresh() are not counted.)
        if need_x and ctx.quantized is not None and ctx.quantized.version != ctx.version:
            raise RuntimeError("the weight's copies were refreshed between forward and backward")
        dy = _unit(dy)
        dx = dw = None
        if need_x and need_w:
            g, g_cols = quantize_both(dy, ctx.seed)
        elif need_x:
            g = quantize(dy, ctx.seed)
        elif need_w:
            g_cols = quantize(dy.t(), ctx.seed)
        if need_x:
            w_cols = MX4._over(w_held, k, n) if ctx.quantized is None else ctx.quantized.cols
            dx = _of_mx4(g, w_cols, dy, ctx.x_dtype, ctx.x_shape)
        if need_w:
            dw = _of_mx4(g_cols, MX4._over(x_held, k, dy.shape[0]), dy, ctx.w_dtype)
        return dx, dw, None, None


def linear(x, weight, quantized=None, seed=None):
    """x weight^T with its gradients, all three products of 4-bit matrices:
    y = Q(x) Q(w)^T, dx = Q(dy) Q(w^T)^T, dw = Q(dy^T) Q(x^T)^T.

    x: [..., K], weight: [N, K], float32 or bfloat16; y and dx have x's type, dw
    weight's.  quantized: the weight's copies where they are kept (a Weight of it, as
    AdamWOptimizer keeps): RuntimeError where they are `behind` it.  seed: round dy
    stochastically, as quantize, another one for every layer and step; None rounds it
    to nearest.  What the backward pass
    keeps of x are 4-bit columns; without gradients (torch.no_grad) none are made.
    Not differentiable twice.  As with all of torch, a
    backward pass is captured in a graph only while no eager graph of the same
    leaves is alive."""
    if weight.dim() != 2 or x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x of shape %s, weight of shape %s" % (tuple(x.shape), tuple(weight.shape)))
    if x.device != weight.device:
        raise ValueError("x on %s, weight on %s" % (x.device, weight.device))
    for t, what in ((x, "x"), (weight, "weight")):
        if t.dtype not in _TYPES:
            raise ValueError("%s must be float32 or bfloat16, not %s" % (what, t.dtype))
        _need_gpu(t, what)
    if quantized is not None and (quantized.rows.shape != tuple(weight.shape)
                                  or quantized.rows.device != weight.device):
        raise ValueError("quantized is of a weight of %d x %d on %s"
                         % (*quantized.rows.shape, quantized.rows.device))
    if quantized is not None and quantized.behind(weight):
        raise RuntimeError("the weight was written or moved since its 4-bit copies were: refresh() "
                           "them")
    if not torch.is_grad_enabled():
        # needs_input_grad would go by requires_grad alone
        m = _unit(x)
        return _forward(x, m, None if _by_rows(m) else quantize(m),
                        quantize(weight) if quantized is None else quantized.rows)
    return _Linear.apply(x, weight, quantized, seed)
