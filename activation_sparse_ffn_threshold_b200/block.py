"""What else a block and its training step need: the linear layer with bias, activation and residual,
the norms before and after a block with its gate and residual scale, and the clipping of gradients.

Calls are checked and marshalled into ``libsfnn.so`` (include/sfnn.h) by ``_block.so``
(csrc/bind/block.cpp) -- native, as their work on the GPU is often shorter than the same in Python.
Tensors lie on one CUDA device, and results belong to the current stream (or to ``stream``, which
the call then runs on).  Autograd follows ``linear`` and ``residual_norm``; the functions with
``_forward`` and ``_backward`` are their passes as plain calls.  What a call writes in place counts as
changed for autograd, as after PyTorch's own operations.
"""
from __future__ import annotations

import importlib.util
import os

import torch
from torch.autograd.function import once_differentiable

from . import _PKG, _check, load_library
from .dense import _err_ptr, _err_ptrs, _follows, _on

__all__ = ["linear", "linear_forward", "linear_backward", "LinearSaved", "residual_norm", "residual_norm_forward",
           "residual_norm_backward", "NormSaved", "clip_grad_norm"]

ACTS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "silu": 3}
NORMS = {None: 0, "none": 0, "rms": 1, "layer": 2}

_native_module = None


def _native():
    """The module _block.so (raises if it was not built)."""
    global _native_module
    if _native_module is None:
        load_library()
        path = os.path.join(_PKG, "_block.so")
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with "
                              f"`python -m activation_sparse_ffn_threshold_b200.build` (nvcc, sm_100a)")
        spec = importlib.util.spec_from_file_location(__package__ + "._block", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native_module = module
    return _native_module


def _err(t) -> int:
    """The error word of t's device (0 for what is no CUDA tensor: the call refuses it)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return 0
    index = t.get_device()
    return _err_ptrs.get(index) or _err_ptr(index)


def _call(stream, t, name, what, *args):
    """A native function's results; ``t`` is on the call's device."""
    f = getattr(_native_module or _native(), name)
    if stream is None:
        got = f(*args)
    else:
        with _on(t.get_device() if isinstance(t, torch.Tensor) and t.is_cuda else stream.device.index, stream):
            got = f(*args)
    if type(got) is int:
        _check(got, what)
    return got


# ------------------------------------------------------------------ linear
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


def linear_forward(x, w, b=None, act=None, residual=None, out_dtype=None, save=False, out=None, stream=None):
    """(y, saved): y = act(x w^T + b) + residual.

    x [..., K], w [N, K], b [N] or None in fp16 or bf16, K a multiple of 8 and rows 16-byte aligned;
    ``act``: None, "relu", "gelu" (z Phi(z)) or "silu".  y [..., N] has the residual's type, x's or
    fp32, or without one ``out_dtype`` (default: x's).  ``out`` takes y, and may be the residual
    itself but share no memory with another input; ``saved`` (with ``save``) goes to
    linear_backward."""
    kind = ACTS.get(act, -1)
    if kind < 0:
        raise ValueError("act must be None, 'relu', 'gelu' or 'silu'")
    y, slopes = _call(stream, x, "linear_forward", "sfnn_linear_forward", x, w, b, kind, residual, out_dtype, save, out,
                      _err(x))
    return y, LinearSaved(x, slopes, kind, y.shape[-1], y.dtype, b is not None) if save else None


def linear_backward(dy, saved: LinearSaved, w, need=(True, True, True), stream=None):
    """(dx, dw, db) from dy [..., N] (of y's type) and a forward pass's ``saved``; those that ``need``
    leaves out, and db without a bias, are None.  The residual's gradient is dy itself."""
    return _call(stream, saved.x, "linear_backward", "sfnn_linear_backward", dy, saved.x, saved.slopes, saved.act, saved.N,
                 saved.y_dtype, saved.has_b, w, tuple(need), _err(saved.x))


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
class NormSaved:
    """What residual_norm_forward keeps for residual_norm_backward: references to its inputs and the
    rows' means and reciprocal deviations."""

    __slots__ = ("tensors", "stats", "options", "dtype")

    def __init__(self, tensors, stats, options, dtype):
        self.tensors, self.stats, self.options, self.dtype = tensors, stats, options, dtype


def _norm_options(pre, post, residual_scale, branch_scale, eps):
    a, b = NORMS.get(pre, -1), NORMS.get(post, -1)
    if a < 0 or b < 0:
        raise ValueError("pre and post must be 'none', 'rms' or 'layer'")
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    return a, b, residual_scale, branch_scale, eps


def residual_norm_forward(x, z=None, pre="rms", w=None, b=None, post="none", post_w=None, post_b=None, gate=None,
                          residual_scale=1.0, branch_scale=1.0, eps=1e-5, dtype=None, save=False, out=None, stream=None):
    """(r, h, saved): r = residual_scale x + branch_scale gate post(z), h = pre(r).

    x [..., d] is the residual stream, z [..., d] (or None: r is x) the block's output, each in
    fp16 or bf16 (h's type: ``dtype``, by default the weights' or the inputs') or fp32; ``pre`` and
    ``post`` are "none", "rms" or "layer", with weights and biases [d] or None; gate is [d], of x's
    shape, or None.  r has x's type, h is None without ``pre``.  ``out`` takes r, and may be x itself
    unless ``save`` but share no memory with another input; ``saved`` goes to residual_norm_backward."""
    options = _norm_options(pre, post, residual_scale, branch_scale, eps)
    r, h, stats, dtype = _call(stream, x, "norm_forward", "sfnn_norm_forward", x, z, gate, w, b, post_w, post_b, *options,
                               dtype, save, out, _err(x))
    return r, h, NormSaved((x, z, gate, w, b, post_w, post_b), stats, options, dtype) if save else None


def residual_norm_backward(dr, dh, saved: NormSaved, need=(True,) * 7, stream=None):
    """(dx, dz, dgate, dw, db, dpost_w, dpost_b) from dr and dh [..., d] (either may be None: zeros);
    those of inputs that were None, and those that ``need`` leaves out, are None."""
    x = saved.tensors[0]
    return _call(stream, x, "norm_backward", "sfnn_norm_backward", *saved.tensors, *saved.options, saved.dtype, saved.stats,
                 dr, dh, tuple(need), _err(x))


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
def clip_grad_norm(grads, max_norm, scale=1.0, out=None, eps=1e-6, stream=None):
    """The norm of all ``grads`` together times ``scale``, as an fp32 tensor of no dimension; the
    gradients become g * scale * min(1, max_norm / (norm + eps)) in place, or in the tensors ``out``.

    grads: CUDA tensors of fp16, bf16 or fp32 in any mix, dense in memory, no memory written twice; ``scale``
    takes a loss scale back out; max_norm = inf leaves them but for ``scale``.  A norm that is not
    finite is returned as it is (an infinite one makes the gradients 0 or NaN, a NaN all of them
    NaN): nothing waits for the device here."""
    grads = list(grads)
    return _call(stream, grads[0] if grads else None, "clip_grad_norm", "sfnn_clip_grad_norm", grads,
                 None if out is None else list(out), max_norm, scale, eps)
