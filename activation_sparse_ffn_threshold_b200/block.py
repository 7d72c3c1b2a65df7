"""What else a block and its training step need: the linear layer with bias, activation and residual,
the norms before and after a block with its gate and residual scale, and the clipping of gradients.

As ``dense``, this module only checks and marshals arguments into ``libsfnn.so``
(include/sfnn.h); tensors lie on one CUDA device, and results belong to the current stream (or to
``stream``, which the call then runs on).  Autograd follows ``linear`` and ``residual_norm``; the
functions with ``_forward`` and ``_backward`` are their passes as plain calls.
"""
from __future__ import annotations

import ctypes
from array import array

import torch
from torch.autograd.function import once_differentiable

from . import BF16, F16, F32, _check, load_library
from .dense import _CODES, _code, _err_ptr, _follows, _mat, _on, _raw_stream, _rows, _same_device, _vp

__all__ = ["linear", "linear_forward", "linear_backward", "LinearSaved", "residual_norm", "residual_norm_forward", "residual_norm_backward", "NormSaved", "clip_grad_norm"]

ACTS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "silu": 3}
NORMS = {None: 0, "none": 0, "rms": 1, "layer": 2}


# ------------------------------------------------------------------ linear
class _LinearDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64), ("b", ctypes.c_void_p)]


class LinearSaved:
    """What linear_forward keeps for linear_backward: a reference to x, and act' (None without an
    activation): a bit per value for a ReLU, 16 bits for the others."""

    __slots__ = ("x", "slopes", "act", "N", "y_dtype", "has_b")

    def __init__(self, x, slopes, act, N, y_dtype, has_b):
        self.x, self.slopes, self.act, self.N, self.y_dtype, self.has_b = x, slopes, act, N, y_dtype, has_b

    @property
    def nbytes(self) -> int:
        """Bytes held, x included."""
        return self.x.numel() * self.x.element_size() + (0 if self.slopes is None else self.slopes.numel())


def _linear_desc(x, w, b, act, y_dtype):
    """(descriptor, N) of a layer's inputs."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    dt = x.dtype
    code = _code(dt)
    px, T, K, ldx = _mat(x, "x", dt)
    pw, N, _, ldw = _mat(w, "w", dt, None, K)
    if not K or K % 8 or not N:
        raise ValueError(f"w must be [N, K] with K a positive multiple of 8, got {tuple(w.shape)}")
    if y_dtype != dt and y_dtype != torch.float32:
        raise TypeError(f"the output is {dt} or fp32, not {y_dtype}")
    index = x.get_device()
    pb = _channels(b, "b", N, dt, index)
    _same_device(index, w)
    return _LinearDesc(T, K, N, code, F32 if y_dtype == torch.float32 else code, act, px, ldx, pw, ldw, pb), N


def linear_forward(x, w, b=None, act=None, residual=None, out_dtype=None, save=False, out=None, stream=None):
    """(y, saved): y = act(x w^T + b) + residual.

    x [..., K], w [N, K], b [N] or None in fp16 or bf16, K a multiple of 8 and rows 16-byte aligned;
    ``act``: None, "relu", "gelu" (z Phi(z)) or "silu".  y [..., N] has the residual's type, x's or
    fp32, or without one ``out_dtype`` (default: x's).  ``out`` takes y and may be the residual itself;
    ``saved`` (with ``save``) goes to linear_backward."""
    if act not in ACTS:
        raise ValueError("act must be None, 'relu', 'gelu' or 'silu'")
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    kind = ACTS[act]
    dt = out_dtype or (x.dtype if residual is None else residual.dtype)
    q, N = _linear_desc(x, w, b, kind, dt)
    index = x.get_device()
    shape = x.shape[:-1] + (N,)
    pr, ldr, py, ldy = None, 0, None, N
    for t, name in ((residual, "residual"), (out, "out")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.dtype != dt or t.shape != shape or t.get_device() != index:
            raise ValueError(f"{name} must be a {dt} tensor of shape {tuple(shape)} on x's device")
        p, r, _, ld = _rows(t, name, N)
        if r and ld < N:
            raise ValueError(f"{name}: rows must not overlap")
        if t is out:
            py, ldy = p, ld
        if t is residual:
            pr, ldr = p, ld
    lib = load_library()
    with _on(index, stream):
        if out is None:
            out = x.new_empty(shape, dtype=dt)
            py = out.data_ptr()
        slopes = None
        if save and kind:
            slopes = x.new_empty(lib.sfnn_linear_slope_bytes(q.T, N, kind), dtype=torch.uint8)
        if q.T:
            nbytes = lib.sfnn_linear_workspace(q.T, q.K, N, 0)
            ws = torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=x.device) if nbytes else None
            _check(lib.sfnn_linear_forward(ctypes.byref(q), pr, ldr, py, ldy, _vp(slopes), _vp(ws), nbytes,
                                           _err_ptr(index), _raw_stream(index)), "sfnn_linear_forward")
    return out, LinearSaved(x, slopes, kind, N, dt, b is not None) if save else None


def linear_backward(dy, saved: LinearSaved, w, need=(True, True, True), stream=None):
    """(dx, dw, db) from dy [..., N] (of y's type) and a forward pass's ``saved``; those that ``need``
    leaves out, and db without a bias, are None.  The residual's gradient is dy itself."""
    x = saved.x
    q, N = _linear_desc(x, w, None, saved.act, saved.y_dtype)
    index = x.get_device()
    if N != saved.N:
        raise ValueError("w must have the forward pass's shape")
    if not isinstance(dy, torch.Tensor) or dy.dtype != saved.y_dtype or dy.shape != x.shape[:-1] + (N,) \
            or dy.get_device() != index:
        raise ValueError(f"dy must be a {saved.y_dtype} tensor of the output's shape on x's device")
    pdy, r, _, lddy = _rows(dy, "dy", N)
    if r and lddy < N:
        raise ValueError("dy: rows must not overlap")
    lib = load_library()
    with _on(index, stream):
        dx = _like(x) if need[0] else None
        dw = _like(w) if need[1] else None
        db = x.new_empty(N) if need[2] and saved.has_b else None
        nbytes = lib.sfnn_linear_workspace(q.T, q.K, N, 1)
        ws = torch.empty_strided((max(16, nbytes),), (1,), dtype=torch.uint8, device=x.device)
        _check(lib.sfnn_linear_backward(ctypes.byref(q), _vp(saved.slopes), pdy, lddy, _vp(dx), _vp(dw), _vp(db),
                                        ws.data_ptr(), nbytes, _err_ptr(index), _raw_stream(index)),
               "sfnn_linear_backward")
    return dx, dw, db


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, residual, act, out_dtype):
        y, saved = linear_forward(x, w, b, act, residual, out_dtype, save=True)
        ctx.save_for_backward(x, w, saved.slopes)
        ctx.rest = saved.act, saved.N, saved.y_dtype, saved.has_b
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, slopes = ctx.saved_tensors
        dx = dw = db = None
        need = ctx.needs_input_grad
        if any(need[:3]):
            dx, dw, db = linear_backward(_even_rows(dy), LinearSaved(x, slopes, *ctx.rest), w, need=need[:3])
        return dx, dw, db, dy if need[3] else None, None, None


def linear(x, w, b=None, act=None, residual=None, out_dtype=None):
    """y of linear_forward, differentiable (once, in reverse mode)."""
    if not _follows(x, w, b, residual):
        return linear_forward(x, w, b, act, residual, out_dtype)[0]
    return _Linear.apply(x, w, b, residual, act, out_dtype)


# ------------------------------------------------------------------ norms
class _NormDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("z_dtype", ctypes.c_int32), ("pre", ctypes.c_int32), ("post", ctypes.c_int32), ("eps", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("branch_scale", ctypes.c_float),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("z", ctypes.c_void_p), ("ldz", ctypes.c_int64),
                ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("w", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("post_w", ctypes.c_void_p), ("post_b", ctypes.c_void_p)]


class NormSaved:
    """What residual_norm_forward keeps for residual_norm_backward: references to its inputs and the
    rows' means and reciprocal deviations."""

    __slots__ = ("tensors", "stats", "options", "dtype")

    def __init__(self, tensors, stats, options, dtype):
        self.tensors, self.stats, self.options, self.dtype = tensors, stats, options, dtype


def _like(t, dtype=None):
    """An uninitialised contiguous tensor of t's shape, in its type or another."""
    return torch.empty_like(t, dtype=dtype) if t.is_contiguous() else t.new_empty(t.shape, dtype=dtype)


def _value_rows(t, name, d, dtype, like=None):
    """(pointer, rows, row stride, type code) of values [..., d] of ``dtype`` (None: no matter) or fp32."""
    p, r, c, ld = _rows(t, name, d)
    dt = t.dtype
    if dt == torch.float32:
        code = F32
    else:
        code = _CODES.get(dt)
        if code is None or (dtype is not None and dt != dtype):
            raise TypeError(f"{name} must be a tensor of fp32 or {dtype or 'fp16 or bf16'}, got {dt}")
    if ld < c and r:
        raise ValueError(f"{name}: rows must not overlap")
    if like is not None and t.shape != like.shape:
        raise ValueError(f"{name} must have the shape {tuple(like.shape)}, got {tuple(t.shape)}")
    return p, r, ld, code


def _channels(t, name, d, dtype, index):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != (d,) or not t.is_contiguous() \
            or t.get_device() != index:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {d} elements on the others' device")
    return t.data_ptr()


def _norm_desc(tensors, options, dtype):
    """(descriptor, 16-bit type) of a call's inputs."""
    x, z, gate, w, b, post_w, post_b = tensors
    pre, post, residual_scale, branch_scale, eps = options
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    for t in (w, x, z, gate, b, post_w, post_b):  # the 16-bit type is the first one's that has it
        if dtype is not None:
            break
        if t is not None and t.dtype != torch.float32:
            dtype = t.dtype
    if dtype is None:
        if pre:
            raise TypeError("dtype (fp16 or bf16) must be given where x, z and the weights do not tell it")
        dtype = torch.float16
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"the norms give fp16 or bf16, not {dtype}")
    d, index = x.shape[-1], x.get_device()
    px, T, ldx, xc = _value_rows(x, "x", d, dtype)
    pz, ldz, zc = None, 0, xc
    if z is not None:
        pz, _, ldz, zc = _value_rows(z, "z", d, dtype, x)
    elif post or gate is not None or not pre or residual_scale != 1.0:
        raise ValueError("without z there is neither a post norm, a gate nor a residual scale, and a pre norm must be given")
    pg, ldg = None, 0
    if gate is not None:
        if isinstance(gate, torch.Tensor) and gate.dim() == 1:
            pg = _channels(gate, "gate", d, dtype, index)
        else:
            if not isinstance(gate, torch.Tensor) or gate.dtype != dtype:
                raise TypeError(f"gate must be a CUDA tensor of {dtype}")
            pg, _, ldg, _ = _value_rows(gate, "gate", d, dtype, x)
    if (not pre and (w is not None or b is not None)) or (not post and (post_w is not None or post_b is not None)):
        raise ValueError("weights are given for a norm that is not there")
    if not 1 <= d <= 32768:
        raise ValueError(f"the norms take rows of 1 to 32768 values, got {d}")
    _same_device(index, z, gate)
    return _NormDesc(T, d, code, xc, zc, pre, post, eps, residual_scale, branch_scale, px, ldx, pz, ldz, pg, ldg,
                     _channels(w, "w", d, dtype, index), _channels(b, "b", d, dtype, index),
                     _channels(post_w, "post_w", d, dtype, index), _channels(post_b, "post_b", d, dtype, index)), dtype


def _norm_options(pre, post, residual_scale, branch_scale, eps):
    if pre not in NORMS or post not in NORMS:
        raise ValueError("pre and post must be 'none', 'rms' or 'layer'")
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    return NORMS[pre], NORMS[post], float(residual_scale), float(branch_scale), float(eps)


def residual_norm_forward(x, z=None, pre="rms", w=None, b=None, post="none", post_w=None, post_b=None, gate=None,
                          residual_scale=1.0, branch_scale=1.0, eps=1e-5, dtype=None, save=False, out=None, stream=None):
    """(r, h, saved): r = residual_scale x + branch_scale gate post(z), h = pre(r).

    x [..., d] is the residual stream, z [..., d] (or None: r is x) the block's output, each in
    fp16 or bf16 (h's type: ``dtype``, by default the weights' or the inputs') or fp32; ``pre`` and
    ``post`` are "none", "rms" or "layer", with weights and biases [d] or None; gate is [d], of x's
    shape, or None.  r has x's type, h is None without ``pre``.  ``out`` takes r, and may be x itself
    unless ``save``; ``saved`` goes to residual_norm_backward."""
    tensors, options = (x, z, gate, w, b, post_w, post_b), _norm_options(pre, post, residual_scale, branch_scale, eps)
    q, dt = _norm_desc(tensors, options, dtype)
    index = x.get_device()
    pr, ldr = None, 0
    if out is not None:
        if z is None:
            raise ValueError("without z nothing is written to out: r is x")
        pr, _, ldr, code = _value_rows(out, "out", q.d, dt, x)
        if code != q.x_dtype or out.get_device() != index:
            raise ValueError("out must be a tensor of x's type on its device")
        if save and pr == q.x:
            raise ValueError("x is needed by the backward pass: out must not be x")
    with _on(index, stream):
        r = x if z is None else out
        if r is None:
            r = _like(x)
            pr, ldr = r.data_ptr(), q.d
        h = _like(x, dt) if q.pre else None
        stats = x.new_empty((q.T, 4), dtype=torch.float32) if save else None
        _check(load_library().sfnn_norm_forward(ctypes.byref(q), pr, ldr, _vp(h), q.d, _vp(stats), _err_ptr(index),
                                                _raw_stream(index)), "sfnn_norm_forward")
    return r, h, NormSaved(tensors, stats, options, dt) if save else None


def residual_norm_backward(dr, dh, saved: NormSaved, need=(True,) * 7, stream=None):
    """(dx, dz, dgate, dw, db, dpost_w, dpost_b) from dr and dh [..., d] (either may be None: zeros);
    those of inputs that were None, and those that ``need`` leaves out, are None."""
    x, z, gate, w, b, post_w, post_b = saved.tensors
    q, dt = _norm_desc(saved.tensors, saved.options, saved.dtype)
    index, d, T = x.get_device(), q.d, q.T
    pdr, lddr, pdh, lddh = None, 0, None, 0
    if dr is not None:
        pdr, _, lddr, code = _value_rows(dr, "dr", d, dt, x)
        if code != q.x_dtype:
            raise TypeError(f"dr must be a tensor of {x.dtype}")
    if dh is not None:
        if not q.pre:
            raise ValueError("the forward pass made no h")
        pdh, _, lddh, code = _value_rows(dh, "dh", d, dt, x)
        if code != q.dtype:
            raise TypeError(f"dh must be a tensor of {dt}")
    for t in (dr, dh):
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must be on one device")
    lib = load_library()
    with _on(index, stream):
        dx, dz, dgate, dw, db, dpw, dpb = [_like(t) if n and t is not None else None
                                           for n, t in zip(need, saved.tensors)]
        nbytes = lib.sfnn_norm_workspace(T, d)
        ws = torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=x.device)
        _check(lib.sfnn_norm_backward(ctypes.byref(q), _vp(saved.stats), pdr, lddr, pdh, lddh, _vp(dx), _vp(dz),
                                      _vp(dgate), _vp(dw), _vp(db), _vp(dpw), _vp(dpb), ws.data_ptr(), nbytes,
                                      _err_ptr(index), _raw_stream(index)), "sfnn_norm_backward")
    return dx, dz, dgate, dw, db, dpw, dpb


def _even_rows(t):
    """A gradient as rows that lie evenly apart and do not overlap (autograd hands out expanded ones)."""
    if t is None or t.is_contiguous():
        return t
    return t.contiguous()


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, gate, w, b, post_w, post_b, options, dtype):
        pre, post, residual_scale, branch_scale, eps = options
        r, h, saved = residual_norm_forward(x, z, pre, w, b, post, post_w, post_b, gate, residual_scale, branch_scale,
                                            eps, dtype, save=True)
        ctx.save_for_backward(x, z, gate, w, b, post_w, post_b, saved.stats)
        ctx.options, ctx.dtype, ctx.parts = saved.options, saved.dtype, (z is not None, h is not None)
        ctx.set_materialize_grads(False)
        return (r, h) if z is not None and h is not None else r if h is None else h

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        *tensors, stats = ctx.saved_tensors
        has_z, has_h = ctx.parts
        dr, dh = grads if has_z and has_h else (None, grads[0]) if has_h else (grads[0], None)
        saved = NormSaved(tuple(tensors), stats, ctx.options, ctx.dtype)
        return residual_norm_backward(_even_rows(dr), _even_rows(dh), saved, need=ctx.needs_input_grad[:7]) + (None, None)


def residual_norm(x, z=None, pre="rms", w=None, b=None, post="none", post_w=None, post_b=None, gate=None,
                  residual_scale=1.0, branch_scale=1.0, eps=1e-5, dtype=None):
    """(r, h) of residual_norm_forward, differentiable (once, in reverse mode)."""
    if not _follows(x, z, gate, w, b, post_w, post_b):
        return residual_norm_forward(x, z, pre, w, b, post, post_w, post_b, gate, residual_scale, branch_scale, eps,
                                     dtype)[:2]
    _norm_options(pre, post, residual_scale, branch_scale, eps)
    got = _ResidualNorm.apply(x, z, gate, w, b, post_w, post_b, (pre, post, residual_scale, branch_scale, eps), dtype)
    return got if isinstance(got, tuple) else (x, got) if z is None else (got, None)


# ------------------------------------------------------------------ clipping
_GRAD_CODES = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}


def _dense(t) -> bool:
    """Whether t's values lie without gaps, in some order of its dimensions."""
    n = 1
    for stride, size in sorted((s, k) for s, k in zip(t.stride(), t.shape) if k != 1):
        if stride != n:
            return False
        n *= size
    return True


def _grad_table(grads, outs, n):
    """The entries of sfnn_grad, four words a tensor; None if something is not a CUDA tensor."""
    T = torch.Tensor
    where = set(map(T.get_device, grads))
    if len(where) != 1 or not grads[0].is_cuda:
        return None
    dtypes = list(map(T.dtype.__get__, grads))
    codes = list(map(_GRAD_CODES.get, dtypes))
    if None in codes:
        bad = dtypes[codes.index(None)]
        raise TypeError(f"gradients are fp16, bf16 or fp32, got {bad}")
    in_order = list(map(T.is_contiguous, grads))
    sizes = list(map(T.numel, grads))
    if not all(in_order) and not all(c or _dense(g) for c, g in zip(in_order, grads)):
        raise ValueError("a gradient's values must lie without gaps")
    table = array("q", bytes(32 * n))
    ptrs = array("q", map(T.data_ptr, grads))
    table[0::4] = table[1::4] = ptrs
    table[2::4] = array("q", sizes)
    table[3::4] = array("q", codes)
    if outs is not grads:
        if set(map(T.get_device, outs)) != where:
            return None
        same = list(map(T.dtype.__get__, outs)) == dtypes and list(map(T.numel, outs)) == sizes
        if same and not (all(in_order) and all(map(T.is_contiguous, outs))):
            same = all(o.shape == g.shape and (o.stride() == g.stride() or c and o.is_contiguous())
                       for g, o, c in zip(grads, outs, in_order))
        if not same:
            raise ValueError("each output must have its gradient's type, size and order of values")
        table[1::4] = array("q", map(T.data_ptr, outs))
    return table


def clip_grad_norm(grads, max_norm, scale=1.0, out=None, eps=1e-6, stream=None):
    """The norm of all ``grads`` together times ``scale``, as an fp32 tensor of no dimension; the
    gradients become g * scale * min(1, max_norm / (norm + eps)) in place, or in the tensors ``out``.

    grads: CUDA tensors of fp16, bf16 or fp32 in any mix, dense in memory, none twice; ``scale``
    takes a loss scale back out; max_norm = inf leaves them but for ``scale``.  A norm that is not
    finite is returned as it is (an infinite one makes the gradients 0 or NaN, a NaN all of them
    NaN): nothing waits for the device here."""
    grads = list(grads)
    outs = grads if out is None else list(out)
    n = len(grads)
    if not n:
        raise ValueError("there are no gradients")
    if len(outs) != n:
        raise ValueError(f"{n} gradients, but {len(outs)} outputs")
    if not (max_norm >= 0 and eps >= 0 and 0 <= scale < float("inf")):
        raise ValueError("max_norm, scale and eps must not be negative, nor scale infinite")
    # whole lists at a time: a hundred tensors' checks one by one would take longer than the kernels
    try:
        table = _grad_table(grads, outs, n)
    except (AttributeError, TypeError):
        table = None
    if table is None:  # which one it is
        raise TypeError("grads and out must be dense CUDA tensors of fp16, bf16 or fp32 on one device")
    first = grads[0]
    index = first.get_device()
    lib = load_library()
    with _on(index, stream):
        norm = first.new_empty((), dtype=torch.float32)
        nbytes = lib.sfnn_clip_workspace(n)
        ws = first.new_empty(nbytes, dtype=torch.uint8)
        _check(lib.sfnn_clip_grad_norm(table.buffer_info()[0], n, max_norm, scale, eps, norm.data_ptr(), ws.data_ptr(), nbytes,
                                       _raw_stream(index)), "sfnn_clip_grad_norm")
    return norm
