"""The dense operators: the gated FFN with its backward pass, 8-bit activation blocks, MXFP4.

As the rest of the binding, this module only checks and marshals arguments into
``libsfnn.so`` (include/sfnn.h); PyTorch provides memory, streams and the autograd graph.
Tensors are fp16 or bf16 on one CUDA device; results belong to the current stream (or to
``stream``, which the call then runs on).  A bounded device-side wait that runs out is
latched per device and returned by ``dense_error``; the word it is latched in is allocated
by a device's first call, which must not be inside a graph capture.

Autograd follows ``gated_ffn`` alone.  ``gated_ffn_forward`` and ``gated_ffn_backward`` are its two
passes as plain calls; what is quantised (``Act8``, ``Mxfp4``), and what is made from it, carries
no gradient.
"""
from __future__ import annotations

import ctypes

import torch
import torch.autograd.forward_ad as _forward_ad
from torch.autograd.function import once_differentiable

from . import BF16, F16, F32, _check, load_library

__all__ = ["gated_ffn", "gated_ffn_forward", "gated_ffn_backward", "GatedSaved", "quantize_act8", "dequantize_act8",
           "Act8", "dense_error", "quantize_mxfp4", "dequantize_mxfp4", "mxfp4_matmul", "mxfp4_linear", "Mxfp4"]

SAVE = {None: 0, "full": 1, "act8": 2}
ACT8_BLOCK = 64


class _GatedDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("n", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("down_layout", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("w_gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64),
                ("w_up", ctypes.c_void_p), ("ld_up", ctypes.c_int64),
                ("w_down", ctypes.c_void_p), ("ld_down", ctypes.c_int64), ("b", ctypes.c_void_p)]


class _GatedSaved(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("r", ctypes.c_void_p),
                ("u", ctypes.c_void_p), ("ld", ctypes.c_int64), ("r_scales", ctypes.c_void_p),
                ("u_scales", ctypes.c_void_p), ("lds", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("ld_x", ctypes.c_int64), ("x_scales", ctypes.c_void_p), ("lds_x", ctypes.c_int64)]


# ------------------------------------------------------------------ helpers
_err_words: dict[int, torch.Tensor] = {}
_err_ptrs: dict[int, int] = {}


def _err_ptr(index: int) -> int:
    """The device's error word (its address)."""
    p = _err_ptrs.get(index)
    if p is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the first dense call on a device allocates its error word: make one before capturing")
        with torch.inference_mode(False):  # an inference tensor could not be cleared outside that mode
            w = torch.zeros(1, dtype=torch.int32, device=torch.device("cuda", index))
        torch.cuda.synchronize(index)  # zeroed before a call on another stream uses it
        _err_words[index] = w
        p = _err_ptrs[index] = w.data_ptr()
    return p


def dense_error(device=None) -> int:
    """Return and clear the latched device-side status of the dense operators on a device
    (synchronises it): 0, or an ``sfnn_status`` code."""
    device = torch.device(device if device is not None else "cuda")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    w = _err_words.get(device.index)
    if w is None:
        return 0
    torch.cuda.synchronize(device)
    code = int(w.item())
    if code:
        w.zero_()
        torch.cuda.synchronize(device)
    return code


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):  # the same handle without building a Stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream


class _Here:
    """A call on the current device and stream: nothing to switch."""

    def __enter__(self):
        return self

    def __exit__(self, *a):
        pass


class _Place:
    """The device of the call's tensors made current, and the stream that it runs on."""

    __slots__ = ("_d", "_s")

    def __init__(self, index, stream):
        if stream is not None and stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
        self._d = torch.cuda.device(index)
        self._s = torch.cuda.stream(stream)

    def __enter__(self):
        self._d.__enter__()
        self._s.__enter__()
        return self

    def __exit__(self, *a):
        self._s.__exit__(*a)
        self._d.__exit__(*a)


_HERE = _Here()


def _on(index: int, stream):
    if stream is None and _current_device() == index:
        return _HERE
    return _Place(index, stream)


_CODES = {torch.float16: F16, torch.bfloat16: BF16}


def _code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"the dense operators take fp16 or bf16 tensors, got {dtype}")
    return code


_INT_MAX = 0x7fffffff  # of the C entry points' sizes; ctypes would cut a larger one without a word


def _rows(t, name, cols=None):
    """(pointer, rows, cols, row stride) of a tensor [..., cols] whose rows lie evenly apart."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if t.is_contiguous() and shape:
        c = shape[-1]
        r = shape[0] if len(shape) == 2 else (t.numel() // c if c else 0)
        if cols is not None and c != cols:
            raise ValueError(f"{name} must have {cols} columns, got {c}")
        if r > _INT_MAX or c > _INT_MAX:
            raise ValueError(f"{name}: {r} rows of {c} columns do not fit 32 bits")
        return t.data_ptr(), r, c, c
    if len(shape) != 2:
        if not shape:
            raise ValueError(f"{name} must have at least one dimension")
        try:
            t = t.view(-1, shape[-1]) if t.numel() else t.reshape(0, shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: its leading dimensions must be viewable as rows") from None
    r, c = t.shape
    if cols is not None and c != cols:
        raise ValueError(f"{name} must have {cols} columns, got {c}")
    sr, sc = t.stride()
    if r > _INT_MAX or c > _INT_MAX:
        raise ValueError(f"{name}: {r} rows of {c} columns do not fit 32 bits")
    if c > 1 and sc != 1 and r:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return t.data_ptr(), r, c, (sr if r > 1 else c)


def _mat(t, name, dtype, rows=None, cols=None):
    """As _rows, for an operand of the tensor cores: 16-byte aligned rows of one type."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a CUDA tensor of {dtype}")
    p, r, c, ld = _rows(t, name, cols)
    if rows is not None and r != rows:
        raise ValueError(f"{name} must have {rows} rows, got {r}")
    if r and (p % 16 or ld % 8 or ld < c):
        raise ValueError(f"{name}: rows must start on 16-byte boundaries and not overlap")
    return p, r, c, ld


def _same_device(index, *ts):
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must be on one device")


def _vp(t):
    return None if t is None else t.data_ptr()


def _follows(*ts) -> bool:
    """Whether autograd follows one of these: a result without it would lose their gradient or tangent."""
    if torch.is_grad_enabled():
        for t in ts:
            if t is not None and t.requires_grad:
                return True
    return _forward_ad._current_level >= 0 and any(
        t is not None and _forward_ad.unpack_dual(t).tangent is not None for t in ts)


def _like(t):
    """An uninitialised contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


# ------------------------------------------------------------------ act8
def _blocks(cols) -> int:
    return (cols + ACT8_BLOCK - 1) // ACT8_BLOCK


class _Planes:
    """Blocks of 64: codes [T, cols rounded up to 64] of ``esize`` bytes and, behind them in
    the same allocation, their fp32 scales [T, blocks]."""

    __slots__ = ("buf", "at", "T", "nb", "esize")

    def __init__(self, buf, at, T, cols, esize):
        self.buf, self.at, self.T, self.nb, self.esize = buf, at, T, _blocks(cols), esize

    @staticmethod
    def size(T, cols, esize) -> int:
        return T * _blocks(cols) * (ACT8_BLOCK * esize + 4)  # a multiple of 4: the next planes start aligned

    def pointers(self):
        """(codes, codes' row stride, scales, scales' row stride)."""
        p = self.buf.data_ptr() + self.at
        ld = self.nb * ACT8_BLOCK
        return p, ld, p + self.T * ld * self.esize, self.nb

    @property
    def codes(self):
        n = self.T * self.nb * ACT8_BLOCK * self.esize
        c = self.buf[self.at:self.at + n].view(self.T, self.nb * ACT8_BLOCK * self.esize)
        return c if self.esize == 1 else c.view(torch.int16)

    @property
    def scales(self):
        a = self.at + self.T * self.nb * ACT8_BLOCK * self.esize
        return self.buf[a:a + 4 * self.T * self.nb].view(torch.float32).view(self.T, self.nb)


class Act8:
    """Rows held as 8-bit codes with an fp32 scale per 64 values (sfnn_act8_quantize)."""

    __slots__ = ("_p", "shape", "dtype", "relu")

    def __init__(self, planes, shape, dtype, relu):
        self._p, self.shape, self.dtype, self.relu = planes, shape, dtype, relu

    @property
    def codes(self):
        """uint8 [T, cols rounded up to 64]; without ``relu`` the bytes are int8."""
        return self._p.codes

    @property
    def scales(self):
        return self._p.scales

    @property
    def nbytes(self) -> int:
        return self._p.buf.numel()


def quantize_act8(x, relu: bool = False, stream=None) -> Act8:
    """x [..., cols] as 8-bit blocks; with ``relu``, relu(x) (a positive value keeps a positive code)."""
    p, T, cols, ld = _rows(x, "x")
    code = _code(x.dtype)
    if cols < 1:
        raise ValueError("x must have at least one column")
    if ld < cols:
        raise ValueError("x: rows must not overlap")
    index = x.get_device()
    with _on(index, stream):
        q = _Planes(x.new_empty(_Planes.size(T, cols, 1), dtype=torch.uint8), 0, T, cols, 1)
        pc, ldq, ps, lds = q.pointers()
        _check(load_library().sfnn_act8_quantize(p, ld, T, cols, code, 1 if relu else 0, pc, ldq, ps, lds,
                                                 _raw_stream(index)), "sfnn_act8_quantize")
    return Act8(q, tuple(x.shape), x.dtype, bool(relu))


def dequantize_act8(q: Act8, dtype=None, out=None, stream=None):
    """The values that q stands for, [..., cols] in ``dtype`` (default: the quantised tensor's)."""
    dtype = dtype or (out.dtype if out is not None else q.dtype)
    given = out is not None
    code = _code(dtype)
    buf, T = q._p.buf, q._p.T
    pc, ldq, ps, lds = q._p.pointers()
    cols = q.shape[-1]
    index = buf.get_device()
    with _on(index, stream):
        if out is None:
            out = buf.new_empty(q.shape, dtype=dtype)
            ld = cols
        else:
            if out.dtype != dtype or tuple(out.shape) != q.shape or out.get_device() != index:
                raise ValueError(f"out must be a {dtype} tensor of shape {tuple(q.shape)} on {buf.device}")
            _, _, _, ld = _rows(out, "out", cols)
            if ld < cols:
                raise ValueError("out: rows must not overlap")
        _check(load_library().sfnn_act8_restore(pc, ldq, ps, lds, T, cols, 1 if q.relu else 0, code, out.data_ptr(), ld,
                                                _raw_stream(index)), "sfnn_act8_restore")
    if given and not out.is_inference():  # autograd then refuses a backward pass that saved what was there before
        torch.autograd.graph.increment_version(out)
    return out


# ------------------------------------------------------------------ mxfp4
class Mxfp4:
    """Rows held as 4-bit codes with a power of two per 32 values (sfnn_mxfp4_quantize)."""

    __slots__ = ("codes", "scales", "shape", "dtype")

    def __init__(self, codes, scales, shape, dtype):
        self.codes, self.scales, self.shape, self.dtype = codes, scales, shape, dtype

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def quantize_mxfp4(x, stream=None) -> Mxfp4:
    """x [..., K] (K a multiple of 32) as MXFP4 rows."""
    p, R, K, ld = _rows(x, "x")
    code = _code(x.dtype)
    if K % 32 or not K:
        raise ValueError(f"the last dimension must be a positive multiple of 32, got {K}")
    if ld < K:
        raise ValueError("x: rows must not overlap")
    lib = load_library()
    index = x.get_device()
    with _on(index, stream):
        q = x.new_empty((R, K // 2), dtype=torch.uint8)
        s = x.new_empty(lib.sfnn_mxfp4_scale_bytes(R, K), dtype=torch.uint8)
        _check(lib.sfnn_mxfp4_quantize(p, ld, R, K, code, q.data_ptr(), s.data_ptr(), _raw_stream(index)),
               "sfnn_mxfp4_quantize")
    return Mxfp4(q, s, x.shape, x.dtype)


def dequantize_mxfp4(q: Mxfp4, dtype=None, stream=None):
    """The values that q stands for, in ``dtype`` (default: the quantised tensor's)."""
    dtype = dtype or q.dtype
    code = _code(dtype)
    K = q.shape[-1]
    index = q.codes.get_device()
    with _on(index, stream):
        out = q.codes.new_empty(q.shape, dtype=dtype)
        _check(load_library().sfnn_mxfp4_restore(q.codes.data_ptr(), q.scales.data_ptr(), q.codes.shape[0], K, code,
                                                 out.data_ptr(), K, _raw_stream(index)), "sfnn_mxfp4_restore")
    return out


def _mx_out(K, w, out_dtype, index):
    """(N, the output's type code) of a product with w."""
    if not isinstance(w, Mxfp4) or len(w.shape) != 2 or not w.shape[0]:
        raise TypeError("w must be an Mxfp4 of a matrix [N, K]")
    N, wk = w.shape
    if K != wk:
        raise ValueError(f"x has {K} columns, w {wk}")
    if w.codes.get_device() != index:
        raise ValueError("all tensors must be on one device")
    return N, F32 if out_dtype == torch.float32 else _code(out_dtype)


def mxfp4_matmul(x: Mxfp4, w: Mxfp4, out_dtype=None, stream=None):
    """x w^T for x [..., K] and w [N, K], both MXFP4; ``out_dtype`` (fp16, bf16 or fp32)
    defaults to the tensor's that x was quantised from."""
    dt = out_dtype or x.dtype
    index = x.codes.get_device()
    K = x.shape[-1]
    N, code = _mx_out(K, w, dt, index)
    with _on(index, stream):
        y = x.codes.new_empty(x.shape[:-1] + (N,), dtype=dt)
        _check(load_library().sfnn_mxfp4_product(x.codes.data_ptr(), x.scales.data_ptr(), x.codes.shape[0],
                                                 w.codes.data_ptr(), w.scales.data_ptr(), N, K, y.data_ptr(), N, code,
                                                 _err_ptr(index), _raw_stream(index)), "sfnn_mxfp4_product")
    return y


class _NoGradient(torch.autograd.Function):
    """A call whose result remembers that it followed from x, and says so instead of ending x's gradient."""

    @staticmethod
    def forward(ctx, x, call, name, *args):
        ctx.name = name
        return call(x, *args)  # (autograd is off in here)

    @staticmethod
    def backward(ctx, dy):
        raise RuntimeError(f"{ctx.name} has no gradient: call it on x.detach() or under torch.no_grad()")


def mxfp4_linear(x, w: Mxfp4, out_dtype=None, stream=None):
    """A linear layer with MXFP4 weights: x [..., K] in fp16 or bf16 is quantised by the call.
    It has no gradient: a backward pass that reaches it raises."""
    p, T, K, ld = _rows(x, "x")
    if (x.requires_grad or _forward_ad._current_level >= 0) and _follows(x):
        return _NoGradient.apply(x, mxfp4_linear, "mxfp4_linear", w, out_dtype, stream)
    dt = x.dtype
    xcode = _code(dt)
    if out_dtype is not None:
        dt = out_dtype
    index = x.get_device()
    N, code = _mx_out(K, w, dt, index)
    if ld < K:
        raise ValueError("x: rows must not overlap")
    lib = load_library()
    with _on(index, stream):
        y = x.new_empty(x.shape[:-1] + (N,), dtype=dt)
        nbytes = lib.sfnn_mxfp4_linear_workspace(T, K)
        ws = x.new_empty(nbytes, dtype=torch.uint8) if nbytes else None  # held until the call is queued
        _check(lib.sfnn_mxfp4_linear(p, ld, T, xcode, w.codes.data_ptr(), w.scales.data_ptr(), N, K, y.data_ptr(), N, code,
                                     None if ws is None else ws.data_ptr(), nbytes, _err_ptr(index),
                                     _raw_stream(index)), "sfnn_mxfp4_linear")
    return y


# ------------------------------------------------------------------ gated FFN
class GatedSaved:
    """What gated_ffn_forward keeps for gated_ffn_backward: relu(G) and U as 16-bit codes and
    X itself ("full"), or everything as 8-bit blocks ("act8"); see sfnn_gated_saved."""

    __slots__ = ("kind", "x", "_buf", "_c", "_dims", "_plan", "shape", "dtype", "has_b")

    def __init__(self, kind, x, T, d, n, has_b):
        self.kind, self.shape, self.dtype, self.has_b = kind, x.shape, x.dtype, has_b
        full = kind == "full"
        e = 2 if full else 1
        nb, db = (n + 63) >> 6, 0 if full else (d + 63) >> 6
        codes = T * nb * 64 * e
        size = (codes + T * nb * 4 + 15) & ~15  # each plane (codes, then scales) on 16 bytes
        nbytes = 2 * size + T * db * 68
        self._dims, self._plan = (T, d, n, e, size), (nb, db, codes, nbytes)
        self._bind(x.new_empty(nbytes, dtype=torch.uint8), x if full else None)

    def _bind(self, buf, x):
        """Take ``buf`` as the memory of the codes and scales, and x."""
        self._buf, self.x = buf, x
        T, _, _, _, size = self._dims
        nb, db, codes, _ = self._plan
        p = buf.data_ptr()
        if db:
            q = p + 2 * size
            self._c = _GatedSaved(2, 0, p, p + size, nb * 64, p + codes, p + size + codes, nb, q, db * 64,
                                  q + T * db * 64, db)
        else:
            self._c = _GatedSaved(1, 0, p, p + size, nb * 64, p + codes, p + size + codes, nb)

    def _release(self):
        """Its tensors, which it holds no longer."""
        tensors = [self._buf] if self.x is None else [self._buf, self.x]
        self._buf = self.x = self._c = None
        return tensors

    def _with(self, buf, x=None):
        """A copy of a released one that holds these (which may come from a hook)."""
        if buf.dtype != torch.uint8 or buf.numel() != self._plan[3] or not buf.is_contiguous() or buf.data_ptr() % 16:
            raise ValueError("the saved activations did not come back as they were")
        s = GatedSaved.__new__(GatedSaved)
        s.kind, s.shape, s.dtype, s.has_b = self.kind, self.shape, self.dtype, self.has_b
        s._dims, s._plan = self._dims, self._plan
        s._bind(buf, x)
        return s

    def _planes(self, i):
        T, d, n, e, size = self._dims
        return _Planes(self._buf, i * size, T, d if i == 2 else n, 1 if i == 2 else e)

    r = property(lambda self: self._planes(0).codes, doc="codes of relu(G): int16 (the bits of a uint16) or uint8")
    u = property(lambda self: self._planes(1).codes, doc="codes of U: int16, or uint8 (the bits of an int8)")
    r_scales = property(lambda self: self._planes(0).scales)
    u_scales = property(lambda self: self._planes(1).scales)
    x_codes = property(lambda self: None if self.kind == "full" else self._planes(2).codes)
    x_scales = property(lambda self: None if self.kind == "full" else self._planes(2).scales)

    @property
    def nbytes(self) -> int:
        """Bytes held, X of "full" included."""
        return self._buf.numel() + (0 if self.x is None else self.x.numel() * self.x.element_size())


def _weights(dtype, w_gate, w_up, w_down, d):
    """(n, and the descriptor's six fields of the weights)."""
    pg, n, d, lg = _mat(w_gate, "w_gate", dtype, None, d)
    pu, _, _, lu = _mat(w_up, "w_up", dtype, n, d)
    pd, _, _, ld = _mat(w_down, "w_down", dtype, d, n)
    if d % 8 or n % 8 or not d or not n:
        raise ValueError(f"d and n must be positive multiples of 8, got d = {d}, n = {n}")
    return n, (pg, lg, pu, lu, pd, ld)


def gated_ffn_forward(x, w_gate, w_up, w_down, b=None, save=None, stream=None):
    """(y, saved): y = (relu(x w_gate^T + b) * (x w_up^T)) w_down^T over all neurons.

    x [..., d]; w_gate, w_up [n, d]; w_down [d, n]; b [n] or None; fp16 or bf16, d and n
    multiples of 8, rows 16-byte aligned (any even row stride).  ``save``: None (saved is
    None), "full" (relu(G) and U as 16-bit codes, a reference to x) or "act8" (all three as
    8-bit blocks)."""
    if save not in SAVE:
        raise ValueError("save must be None, 'full' or 'act8'")
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    dt = x.dtype
    code = _code(dt)
    px, T, d, ldx = _mat(x, "x", dt)
    n, wf = _weights(dt, w_gate, w_up, w_down, d)
    pb = None
    if b is not None:
        if b.dtype != dt or b.shape != (n,) or not b.is_contiguous():
            raise ValueError(f"b must be a contiguous {dt} tensor of {n} elements")
        pb = b.data_ptr()
    index = x.get_device()
    _same_device(index, w_gate, w_up, w_down, b)
    lib = load_library()
    with _on(index, stream):
        y = _like(x)
        saved = csaved = None
        if save is not None:
            saved = GatedSaved(save, x, T, d, n, b is not None)
            csaved = ctypes.byref(saved._c)
        if T:
            nbytes = lib.sfnn_gated_workspace(T, d, n, 0)
            ws = x.new_empty(nbytes, dtype=torch.uint8)
            q = _GatedDesc(T, d, n, code, 0, 0, px, ldx, *wf, pb)
            _check(lib.sfnn_gated_forward(ctypes.byref(q), y.data_ptr(), d, code, csaved, ws.data_ptr(), nbytes,
                                          _err_ptr(index), _raw_stream(index)), "sfnn_gated_forward")
    return y, saved


def gated_ffn_backward(dy, saved: GatedSaved, w_gate, w_up, w_down, need=(True, True, True, True, True), stream=None):
    """(dx, dw_gate, dw_up, dw_down, db) from dy [..., d] and a forward pass's ``saved``; those
    that ``need`` leaves out, and db without a bias, are None."""
    dt = saved.dtype
    d = saved.shape[-1]
    pdy, T, _, lddy = _mat(dy, "dy", dt, None, d)
    n, wf = _weights(dt, w_gate, w_up, w_down, d)
    full = saved.kind == "full"
    if dy.shape != saved.shape or saved._dims[2] != n:
        raise ValueError("dy and the weights must have the forward pass's shapes")
    px, ldx = None, 0
    if full:
        px, _, _, ldx = _mat(saved.x, "x", dt, T, d)
    index = dy.get_device()
    _same_device(index, w_gate, w_up, w_down, saved._buf)
    lib = load_library()
    with _on(index, stream):
        dx = _like(dy) if need[0] else None
        dwg = _like(w_gate) if need[1] else None
        dwu = _like(w_up) if need[2] else None
        dwd = _like(w_down) if need[3] else None
        db = dy.new_empty(n) if need[4] and saved.has_b else None
        nbytes = lib.sfnn_gated_workspace(T, d, n, 1)
        ws = dy.new_empty(max(16, nbytes), dtype=torch.uint8)
        q = _GatedDesc(T, d, n, _code(dt), 0, 0, px, ldx, *wf, None)
        _check(lib.sfnn_gated_backward(ctypes.byref(q), pdy, lddy, ctypes.byref(saved._c), _vp(dx), _vp(dwg),
                                       _vp(dwu), _vp(dwd), _vp(db), ws.data_ptr(), max(16, nbytes), _err_ptr(index),
                                       _raw_stream(index)), "sfnn_gated_backward")
    return dx, dwg, dwu, dwd, db


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, b, checkpoint):
        y, saved = gated_ffn_forward(x, w_gate, w_up, w_down, b, save=checkpoint)
        # every tensor through autograd, which frees them with the backward pass, hands them to hooks
        # that move them elsewhere, and notices a change in place
        ctx.save_for_backward(w_gate, w_up, w_down, *saved._release())
        ctx.saved = saved
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w_gate, w_up, w_down, *kept = ctx.saved_tensors
        if dy.stride() != torch.empty(dy.shape, device="meta").stride() or dy.data_ptr() % 16:
            dy = dy.contiguous() if not dy.is_contiguous() else dy.clone()
        return gated_ffn_backward(dy, ctx.saved._with(*kept), w_gate, w_up, w_down,
                                  need=ctx.needs_input_grad[:5]) + (None,)


def gated_ffn(x, w_gate, w_up, w_down, b=None, checkpoint: str = "full"):
    """gated_ffn_forward as a differentiable function (once, in reverse mode); ``checkpoint``
    ("full" or "act8") is how the activations are held until the backward pass."""
    if checkpoint not in ("full", "act8"):
        raise ValueError("checkpoint must be 'full' or 'act8'")
    if not _follows(x, w_gate, w_up, w_down, b):
        return gated_ffn_forward(x, w_gate, w_up, w_down, b)[0]
    return _GatedFFN.apply(x, w_gate, w_up, w_down, b, checkpoint)
