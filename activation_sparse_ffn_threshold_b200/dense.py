"""The dense operators: the gated FFN with its backward pass, 8-bit activation blocks, MXFP4.

As the rest of the binding, this module only checks and marshals arguments into
``libsfnn.so`` (include/sfnn.h); PyTorch provides memory, streams and the autograd graph.
Tensors are fp16 or bf16 on one CUDA device; results belong to the current stream (or to
``stream``, which the call then runs on).  A bounded device-side wait that runs out is
latched per device and returned by ``dense_error``.
"""
from __future__ import annotations

import ctypes

import torch
from torch.autograd.function import once_differentiable

from . import BF16, F16, F32, SfnnError, _check, load_library

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


def _err_word(device) -> torch.Tensor:
    w = _err_words.get(device.index)
    if w is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the first dense call on a device allocates its error word: make one before capturing")
        w = torch.zeros(1, dtype=torch.int32, device=device)
        torch.cuda.synchronize(device)  # zeroed before a call on another stream uses it
        _err_words[device.index] = w
    return w


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


class _Place:
    """The device of the call's tensors made current, and the stream that it runs on."""

    __slots__ = ("dev", "stream", "raw", "_d", "_s")

    def __init__(self, device, stream):
        self.dev = device
        self._d = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        self._s = None if stream is None else torch.cuda.stream(stream)
        self.stream = stream

    def __enter__(self):
        if self._d is not None:
            self._d.__enter__()
        if self._s is not None:
            self._s.__enter__()
        self.raw = (self.stream or torch.cuda.current_stream(self.dev)).cuda_stream
        return self

    def __exit__(self, *a):
        if self._s is not None:
            self._s.__exit__(*a)
        if self._d is not None:
            self._d.__exit__(*a)


def _code(dtype) -> int:
    if dtype == torch.float16:
        return F16
    if dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"the dense operators take fp16 or bf16 tensors, got {dtype}")


def _rows(t, name, cols=None):
    """(pointer, rows, cols, row stride) of a tensor [..., cols] whose rows lie evenly apart."""
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{name} must have at least one dimension")
        try:
            t = t.view(-1, t.shape[-1]) if t.numel() else t.reshape(0, t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: its leading dimensions must be viewable as rows") from None
    r, c = t.shape
    if cols is not None and c != cols:
        raise ValueError(f"{name} must have {cols} columns, got {c}")
    sr, sc = t.stride()
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


def _same_device(ts, device):
    for t in ts:
        if t is not None and t.device != device:
            raise ValueError("all tensors must be on one device")


def _vp(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ act8
class Act8:
    """Rows held as 8-bit codes with an fp32 scale per 64 values (sfnn_act8_quantize)."""

    __slots__ = ("codes", "scales", "shape", "dtype", "relu")

    def __init__(self, codes, scales, shape, dtype, relu):
        self.codes, self.scales, self.shape, self.dtype, self.relu = codes, scales, shape, dtype, relu

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scales.numel()


def _act8_empty(T, cols, device):
    nb = (cols + ACT8_BLOCK - 1) // ACT8_BLOCK
    return (torch.empty((T, nb * ACT8_BLOCK), dtype=torch.uint8, device=device),
            torch.empty((T, nb), dtype=torch.float32, device=device))


def quantize_act8(x, relu: bool = False, stream=None) -> Act8:
    """x [..., cols] as 8-bit blocks; with ``relu``, relu(x) (a positive value keeps a positive code)."""
    code = _code(x.dtype) if isinstance(x, torch.Tensor) else 0
    p, T, cols, ld = _rows(x, "x")
    if cols < 1:
        raise ValueError("x must have at least one column")
    if ld < cols:
        raise ValueError("x: rows must not overlap")
    with _Place(x.device, stream) as at:
        q, s = _act8_empty(T, cols, x.device)
        _check(load_library().sfnn_act8_quantize(p, ld, T, cols, code, int(bool(relu)), q.data_ptr(), q.shape[1],
                                                 s.data_ptr(), s.shape[1], at.raw), "sfnn_act8_quantize")
    return Act8(q, s, tuple(x.shape), x.dtype, bool(relu))


def dequantize_act8(q: Act8, dtype=None, out=None, stream=None):
    """The values that q stands for, [..., cols] in ``dtype`` (default: the quantised tensor's)."""
    dtype = dtype or (out.dtype if out is not None else q.dtype)
    code = _code(dtype)
    cols = q.shape[-1]
    T = q.codes.shape[0]
    with _Place(q.codes.device, stream) as at:
        if out is None:
            out = torch.empty(q.shape, dtype=dtype, device=q.codes.device)
        elif out.dtype != dtype or tuple(out.shape) != tuple(q.shape) or out.device != q.codes.device:
            raise ValueError(f"out must be a {dtype} tensor of shape {tuple(q.shape)} on {q.codes.device}")
        p, _, _, ld = _rows(out, "out", cols)
        if ld < cols:
            raise ValueError("out: rows must not overlap")
        _check(load_library().sfnn_act8_restore(q.codes.data_ptr(), q.codes.shape[1], q.scales.data_ptr(),
                                                q.scales.shape[1], T, cols, int(q.relu), code, p, ld, at.raw),
               "sfnn_act8_restore")
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
    code = _code(x.dtype) if isinstance(x, torch.Tensor) else 0
    p, R, K, ld = _rows(x, "x")
    if K % 32 or not K:
        raise ValueError(f"the last dimension must be a positive multiple of 32, got {K}")
    if ld < K:
        raise ValueError("x: rows must not overlap")
    lib = load_library()
    with _Place(x.device, stream) as at:
        q = torch.empty((R, K // 2), dtype=torch.uint8, device=x.device)
        s = torch.empty(lib.sfnn_mxfp4_scale_bytes(R, K), dtype=torch.uint8, device=x.device)
        _check(lib.sfnn_mxfp4_quantize(p, ld, R, K, code, q.data_ptr(), s.data_ptr(), at.raw), "sfnn_mxfp4_quantize")
    return Mxfp4(q, s, tuple(x.shape), x.dtype)


def dequantize_mxfp4(q: Mxfp4, dtype=None, stream=None):
    """The values that q stands for, in ``dtype`` (default: the quantised tensor's)."""
    dtype = dtype or q.dtype
    K = q.shape[-1]
    with _Place(q.codes.device, stream) as at:
        out = torch.empty(q.shape, dtype=dtype, device=q.codes.device)
        _check(load_library().sfnn_mxfp4_restore(q.codes.data_ptr(), q.scales.data_ptr(), q.codes.shape[0], K,
                                                 _code(dtype), out.data_ptr(), K, at.raw), "sfnn_mxfp4_restore")
    return out


def _mx_out(shape, w, out_dtype, device):
    if not isinstance(w, Mxfp4) or len(w.shape) != 2 or not w.shape[0]:
        raise TypeError("w must be an Mxfp4 of a matrix [N, K]")
    if shape[-1] != w.shape[1]:
        raise ValueError(f"x has {shape[-1]} columns, w {w.shape[1]}")
    if w.codes.device != device:
        raise ValueError("all tensors must be on one device")
    return F32 if out_dtype == torch.float32 else _code(out_dtype)


def mxfp4_matmul(x: Mxfp4, w: Mxfp4, out_dtype=None, stream=None):
    """x w^T for x [..., K] and w [N, K], both MXFP4; ``out_dtype`` (fp16, bf16 or fp32)
    defaults to the tensor's that x was quantised from."""
    dt = out_dtype or x.dtype
    dev = x.codes.device
    code = _mx_out(x.shape, w, dt, dev)
    N, K = w.shape
    T = x.codes.shape[0]
    with _Place(dev, stream) as at:
        y = torch.empty(x.shape[:-1] + (N,), dtype=dt, device=dev)
        _check(load_library().sfnn_mxfp4_product(x.codes.data_ptr(), x.scales.data_ptr(), T, w.codes.data_ptr(),
                                                 w.scales.data_ptr(), N, K, y.data_ptr(), N, code,
                                                 _err_word(dev).data_ptr(), at.raw), "sfnn_mxfp4_product")
    return y


def mxfp4_linear(x, w: Mxfp4, out_dtype=None, stream=None):
    """A linear layer with MXFP4 weights: x [..., K] in fp16 or bf16 is quantised by the call."""
    dt = out_dtype or (x.dtype if isinstance(x, torch.Tensor) else None)
    p, T, K, ld = _rows(x, "x")
    xcode = _code(x.dtype)
    dev = x.device
    code = _mx_out(x.shape, w, dt, dev)
    if ld < K:
        raise ValueError("x: rows must not overlap")
    N = w.shape[0]
    lib = load_library()
    with _Place(dev, stream) as at:
        y = torch.empty(x.shape[:-1] + (N,), dtype=dt, device=dev)
        ws = torch.empty(max(16, lib.sfnn_mxfp4_linear_workspace(T, K)), dtype=torch.uint8, device=dev)
        _check(lib.sfnn_mxfp4_linear(p, ld, T, xcode, w.codes.data_ptr(), w.scales.data_ptr(), N, K, y.data_ptr(), N, code,
                                     ws.data_ptr(), ws.numel(), _err_word(dev).data_ptr(), at.raw), "sfnn_mxfp4_linear")
    return y


# ------------------------------------------------------------------ gated FFN
class GatedSaved:
    """What gated_ffn_forward keeps for gated_ffn_backward: relu(G) and U, and X itself
    ("full") or everything as 8-bit blocks ("act8")."""

    __slots__ = ("kind", "x", "r", "u", "r_scales", "u_scales", "x_codes", "x_scales", "shape", "dtype", "has_b")

    def tensors(self):
        return [t for t in (self.x, self.r, self.u, self.r_scales, self.u_scales, self.x_codes, self.x_scales)
                if t is not None]

    @property
    def nbytes(self) -> int:
        """Bytes held, X of "full" included."""
        return sum(t.numel() * t.element_size() for t in self.tensors())

    def _fill(self):
        c = _GatedSaved()
        c.kind = SAVE[self.kind]
        c.r, c.u, c.ld = _vp(self.r), _vp(self.u), self.r.shape[1]
        if self.kind == "act8":
            c.r_scales, c.u_scales, c.lds = _vp(self.r_scales), _vp(self.u_scales), self.r_scales.shape[1]
            c.x, c.ld_x = _vp(self.x_codes), self.x_codes.shape[1]
            c.x_scales, c.lds_x = _vp(self.x_scales), self.x_scales.shape[1]
        return c


def _weights(desc, dtype, w_gate, w_up, w_down, d=None):
    desc.w_gate, n, d, desc.ld_gate = _mat(w_gate, "w_gate", dtype, None, d)
    desc.w_up, _, _, desc.ld_up = _mat(w_up, "w_up", dtype, n, d)
    desc.w_down, _, _, desc.ld_down = _mat(w_down, "w_down", dtype, d, n)
    if d % 8 or n % 8 or not d or not n:
        raise ValueError(f"d and n must be positive multiples of 8, got d = {d}, n = {n}")
    desc.d, desc.n, desc.dtype = d, n, _code(dtype)
    return n, d


def gated_ffn_forward(x, w_gate, w_up, w_down, b=None, save=None, stream=None):
    """(y, saved): y = (relu(x w_gate^T + b) * (x w_up^T)) w_down^T over all neurons.

    x [..., d]; w_gate, w_up [n, d]; w_down [d, n]; b [n] or None; fp16 or bf16, d and n
    multiples of 8, rows 16-byte aligned (any even row stride).  ``save``: None (saved is
    None), "full" (relu(G), U and a reference to x) or "act8" (all three as 8-bit blocks)."""
    if save not in SAVE:
        raise ValueError("save must be None, 'full' or 'act8'")
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise TypeError("x must be a CUDA tensor")
    dt = x.dtype
    code = _code(dt)
    q = _GatedDesc()
    q.x, T, d, q.ldx = _mat(x, "x", dt)
    n, d = _weights(q, dt, w_gate, w_up, w_down, d)
    q.T = T
    if b is not None:
        if b.dtype != dt or tuple(b.shape) != (n,) or not b.is_contiguous():
            raise ValueError(f"b must be a contiguous {dt} tensor of {n} elements")
        q.b = b.data_ptr()
    dev = x.device
    _same_device((w_gate, w_up, w_down, b), dev)
    lib = load_library()
    with _Place(dev, stream) as at:
        y = torch.empty(x.shape, dtype=dt, device=dev)
        saved = csaved = None
        if save is not None:
            saved = GatedSaved()
            saved.kind, saved.shape, saved.dtype, saved.has_b = save, tuple(x.shape), dt, b is not None
            saved.x = saved.r_scales = saved.u_scales = saved.x_codes = saved.x_scales = None
            if save == "full":
                saved.x = x
                ru = torch.empty((2, T, n), dtype=dt, device=dev)
                saved.r, saved.u = ru[0], ru[1]
            else:
                saved.r, saved.r_scales = _act8_empty(T, n, dev)
                saved.u, saved.u_scales = _act8_empty(T, n, dev)
                saved.x_codes, saved.x_scales = _act8_empty(T, d, dev)
            csaved = ctypes.byref(saved._fill())
        if T:
            ws = torch.empty(lib.sfnn_gated_workspace(T, d, n, 0), dtype=torch.uint8, device=dev)
            _check(lib.sfnn_gated_forward(ctypes.byref(q), y.data_ptr(), d, code, csaved, ws.data_ptr(), ws.numel(),
                                          _err_word(dev).data_ptr(), at.raw), "sfnn_gated_forward")
    return y, saved


def gated_ffn_backward(dy, saved: GatedSaved, w_gate, w_up, w_down, need=(True, True, True, True, True), stream=None):
    """(dx, dw_gate, dw_up, dw_down, db) from dy [..., d] and a forward pass's ``saved``; those
    that ``need`` leaves out, and db without a bias, are None."""
    dt = saved.dtype
    q = _GatedDesc()
    d = saved.shape[-1]
    pdy, T, _, lddy = _mat(dy, "dy", dt, None, d)
    n, d = _weights(q, dt, w_gate, w_up, w_down, d)
    if tuple(dy.shape) != saved.shape or saved.r.shape[1] != (n if saved.kind == "full" else -(-n // 64) * 64):
        raise ValueError("dy and the weights must have the forward pass's shapes")
    q.T = T
    if saved.kind == "full":
        q.x, _, _, q.ldx = _mat(saved.x, "x", dt, T, d)
    dev = dy.device
    _same_device((w_gate, w_up, w_down, saved.r), dev)
    lib = load_library()
    with _Place(dev, stream) as at:
        def out(on, *shape):
            return torch.empty(shape, dtype=dt, device=dev) if on else None
        dx = torch.empty(dy.shape, dtype=dt, device=dev) if need[0] else None
        dwg, dwu, dwd = out(need[1], n, d), out(need[2], n, d), out(need[3], d, n)
        db = out(need[4] and saved.has_b, n)
        ws = torch.empty(max(16, lib.sfnn_gated_workspace(T, d, n, 1)), dtype=torch.uint8, device=dev)
        _check(lib.sfnn_gated_backward(ctypes.byref(q), pdy, lddy, ctypes.byref(saved._fill()), _vp(dx), _vp(dwg),
                                       _vp(dwu), _vp(dwd), _vp(db), ws.data_ptr(), ws.numel(),
                                       _err_word(dev).data_ptr(), at.raw), "sfnn_gated_backward")
    return dx, dwg, dwu, dwd, db


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, b, checkpoint):
        y, saved = gated_ffn_forward(x, w_gate, w_up, w_down, b, save=checkpoint)
        ctx.saved = saved
        keep = [w_gate, w_up, w_down]
        if saved.x is not None:  # through autograd, which notices a change in place
            keep.append(saved.x)
            saved.x = None
        ctx.save_for_backward(*keep)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w_gate, w_up, w_down, *x = ctx.saved_tensors
        saved = ctx.saved
        if dy.stride() != torch.empty(dy.shape, device="meta").stride() or dy.data_ptr() % 16:
            dy = dy.contiguous() if not dy.is_contiguous() else dy.clone()
        if x:
            full = GatedSaved()
            for k in GatedSaved.__slots__:
                setattr(full, k, getattr(saved, k))
            full.x = x[0]
            saved = full
        return gated_ffn_backward(dy, saved, w_gate, w_up, w_down, need=ctx.needs_input_grad[:5]) + (None,)


def gated_ffn(x, w_gate, w_up, w_down, b=None, checkpoint: str = "full"):
    """gated_ffn_forward as a differentiable function; ``checkpoint`` ("full" or "act8") is
    how the activations are held until the backward pass."""
    if checkpoint not in ("full", "act8"):
        raise ValueError("checkpoint must be 'full' or 'act8'")
    if not torch.is_grad_enabled() or not any(t is not None and t.requires_grad for t in (x, w_gate, w_up, w_down, b)):
        return gated_ffn_forward(x, w_gate, w_up, w_down, b)[0]
    return _GatedFFN.apply(x, w_gate, w_up, w_down, b, checkpoint)
