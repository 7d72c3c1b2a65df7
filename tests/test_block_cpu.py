"""Refusals of the operators around the products, which need no GPU: the C entry points return a
status and launch nothing, the binding raises."""
import ctypes
import math

import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf


class NormDesc(ctypes.Structure):  # sfnn_norm_desc
    _fields_ = [(k, ctypes.c_int32) for k in ("T", "d", "dtype", "x_dtype", "z_dtype", "pre", "post")] + \
        [(k, ctypes.c_float) for k in ("eps", "residual_scale", "branch_scale")] + \
        [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("z", ctypes.c_void_p), ("ldz", ctypes.c_int64),
         ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64)] + [(k, ctypes.c_void_p) for k in ("w", "b", "post_w", "post_b")]


class LinearDesc(ctypes.Structure):  # sfnn_linear_desc
    _fields_ = [(k, ctypes.c_int32) for k in ("T", "K", "N", "dtype", "y_dtype", "act")] + \
        [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64),
         ("b", ctypes.c_void_p)]


INVALID, UNSUPPORTED = sf.STATUS_CODES["SFNN_ERR_INVALID_ARG"], sf.STATUS_CODES["SFNN_ERR_UNSUPPORTED"]


def norm(T=2, d=64, dtype=sf.F16, **kw):
    q = NormDesc(T, d, dtype, dtype, dtype, 1, 0, 1e-5, 1.0, 1.0, 4096, d, 4096, d, None, 0, 4096, None, None, None)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


NORM_REFUSALS = [
    (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(d=32769), UNSUPPORTED), (dict(T=(1 << 28) + 1), UNSUPPORTED),
    (dict(dtype=sf.F32), INVALID), (dict(x_dtype=sf.BF16), INVALID), (dict(z_dtype=sf.I8), INVALID), (dict(pre=3), INVALID),
    (dict(post=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(x=None), INVALID),
    (dict(x=4097), INVALID), (dict(x_dtype=sf.F32, x=4098), INVALID), (dict(ldx=63), INVALID), (dict(ldz=-64), INVALID),
    (dict(z=None, post=1), INVALID), (dict(z=None, gate=4096), INVALID), (dict(z=None, pre=0), INVALID),
    (dict(z=None, residual_scale=0.5), INVALID), (dict(pre=0), INVALID), (dict(post_w=4096), INVALID),
    (dict(w=4097), INVALID), (dict(gate=4096, ldg=32), INVALID), (dict(gate=4097), INVALID)]


@pytest.mark.parametrize("kw,want", NORM_REFUSALS)
def test_norms_refuse_bad_descriptors(kw, want):
    lib = sf.load_library()
    q = norm(**kw)
    assert lib.sfnn_norm_forward(ctypes.byref(q), 4096, 64, 4096, 64, None, 4096, None) == want
    assert lib.sfnn_norm_backward(ctypes.byref(q), 4096, 4096, 64, None, 64, 4096, None, None, None, None, None, None,
                                  4096, 1 << 40, 4096, None) == want


def test_norms_refuse_bad_buffers():
    lib = sf.load_library()

    def forward(q, r=4096, ldr=64, h=4096, ldh=64, stats=None, err=4096):
        return lib.sfnn_norm_forward(ctypes.byref(q), r, ldr, h, ldh, stats, err, None)
    assert lib.sfnn_norm_forward(None, 4096, 64, 4096, 64, None, 4096, None) == INVALID
    for kw in (dict(r=None), dict(ldr=63), dict(r=4097), dict(h=None), dict(ldh=60), dict(stats=4100), dict(err=None),
               dict(err=4098)):
        assert forward(norm(), **kw) == INVALID, kw
    assert forward(norm(T=0), r=None, h=None) == 0

    def backward(q, stats=4096, dr=4096, lddr=64, dh=4096, lddh=64, dx=4096, dz=4096, dgate=None, dw=4096, db=None, dpw=None,
                 dpb=None, ws=4096, nbytes=1 << 40, err=4096):
        return lib.sfnn_norm_backward(None if q is None else ctypes.byref(q), stats, dr, lddr, dh, lddh, dx, dz, dgate, dw,
                                      db, dpw, dpb, ws, nbytes, err, None)
    assert backward(None) == INVALID
    for kw in (dict(stats=None), dict(stats=4104), dict(err=None), dict(lddr=63), dict(dr=4097), dict(dh=4097), dict(lddh=8), dict(dx=4097),
               dict(dz=4097), dict(dgate=4096), dict(dw=4097), dict(dpw=4096), dict(dpb=4096), dict(ws=None),
               dict(ws=4104), dict(nbytes=8)):
        status = backward(norm(), **kw)
        assert status == INVALID or (status == 2 and kw.keys() & {"ws", "nbytes"}), kw  # (2: no device to size it by)
    assert backward(norm(pre=0, w=None), dw=None) == INVALID and backward(norm(pre=0, w=None), dh=None) == INVALID
    assert backward(norm(z=None)) == INVALID
    assert lib.sfnn_norm_workspace(-1, 64) < 0 and lib.sfnn_norm_workspace(4, 0) < 0
    assert lib.sfnn_norm_workspace(4, 32769) < 0 and lib.sfnn_norm_workspace(0, 64) > 0


def test_clipping_refuses():
    lib = sf.load_library()

    def clip(rows=((4096, 4096, 10, sf.F16),), max_norm=1.0, scale=1.0, eps=1e-6, norm=4096, ws=4096, nbytes=1 << 40, n=None):
        flat = [v for r in rows for v in r]
        return lib.sfnn_clip_grad_norm((ctypes.c_int64 * max(1, len(flat)))(*flat), len(rows) if n is None else n, max_norm,
                                       scale, eps, norm, ws, nbytes, None)
    for kw in (dict(n=-1), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(scale=-1.0), dict(scale=math.inf),
               dict(scale=math.nan), dict(eps=-1.0), dict(norm=None), dict(norm=4098), dict(ws=None), dict(ws=4100),
               dict(nbytes=8)):
        assert clip(**kw) == INVALID, kw
    for row in ((0, 4096, 10, sf.F16), (4096, 0, 10, sf.F16), (4097, 4096, 10, sf.F16), (4096, 4098, 10, sf.F32),
                (4096, 4096, -1, sf.F16), (4096, 4096, 10, sf.I8), (4096, 4106, 10, sf.F16)):
        assert clip(rows=(row,)) == INVALID, row
    assert clip(rows=((4096, 4096, (1 << 40) + 1, sf.F16),)) == UNSUPPORTED
    a, b = (4096, 4096, 10, sf.F16), (4114, 4114, 10, sf.F16)
    assert clip(rows=(a, a)) == INVALID and clip(rows=(a, b)) == INVALID
    assert clip(rows=((4096, 8192, 10, sf.F16), (8192, 9000, 10, sf.F16))) == INVALID
    assert lib.sfnn_clip_grad_norm(None, 1, 1.0, 1.0, 1e-6, 4096, 4096, 1 << 40, None) == INVALID
    assert lib.sfnn_clip_workspace(-1) < 0 and lib.sfnn_clip_workspace(0) > 0


def test_binding_refuses_host_tensors_and_bad_options():
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        sf.residual_norm_forward(x)
    with pytest.raises(TypeError):
        sf.residual_norm(x, x)
    with pytest.raises(ValueError):
        sf.residual_norm_forward(x, pre="batch")
    with pytest.raises(ValueError):
        sf.residual_norm(x, eps=-1.0)
    with pytest.raises(TypeError):
        sf.clip_grad_norm([x], 1.0)
    with pytest.raises(ValueError):
        sf.clip_grad_norm([], 1.0)
    for kw in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(max_norm=1.0, scale=math.inf), dict(max_norm=1.0, eps=-1)):
        with pytest.raises(ValueError):
            sf.clip_grad_norm([x], **kw)
    with pytest.raises(ValueError):
        sf.clip_grad_norm([x], 1.0, out=[])


def linear(T=4, K=64, N=40, dtype=sf.F16, y_dtype=None, act=1, **kw):
    q = LinearDesc(T, K, N, dtype, dtype if y_dtype is None else y_dtype, act, 4096, K, 4096, K, 4096)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(dtype=sf.F32), UNSUPPORTED),
    (dict(dtype=7), INVALID), (dict(y_dtype=sf.BF16), INVALID), (dict(act=4), INVALID), (dict(act=-1), INVALID),
    (dict(K=60), UNSUPPORTED), (dict(K=(1 << 20) + 8), UNSUPPORTED), (dict(N=(1 << 20) + 1), UNSUPPORTED),
    (dict(T=(1 << 24) + 1), UNSUPPORTED), (dict(x=None), INVALID), (dict(x=4104), INVALID), (dict(ldx=60), INVALID),
    (dict(ldx=68), INVALID), (dict(w=None), INVALID), (dict(w=8), INVALID), (dict(ldw=66), INVALID), (dict(b=4097), INVALID)])
def test_linear_refuses_bad_descriptors(kw, want):
    lib = sf.load_library()
    q = linear(**kw)
    assert lib.sfnn_linear_forward(ctypes.byref(q), None, 0, 4096, 40, None, 4096, 1 << 40, 4096, None) == want
    assert lib.sfnn_linear_backward(ctypes.byref(q), 4096, 4096, 40, 4096, 4096, 4096, 4096, 1 << 40, 4096, None) == want


def test_linear_refuses_bad_buffers():
    lib = sf.load_library()

    def forward(q, res=None, ldr=40, y=4096, ldy=40, slopes=None, err=4096):
        return lib.sfnn_linear_forward(None if q is None else ctypes.byref(q), res, ldr, y, ldy, slopes, 4096, 1 << 40, err,
                                       None)
    assert forward(None) == INVALID
    for kw in (dict(y=None), dict(y=4097), dict(ldy=39), dict(res=4097), dict(res=4096, ldr=39), dict(slopes=4100),
               dict(err=None), dict(err=4098)):
        assert forward(linear(), **kw) == INVALID, kw
    assert forward(linear(y_dtype=sf.F32), y=4098) == INVALID and forward(linear(act=0), slopes=4096) == INVALID
    assert forward(linear(T=0), y=None) == 0

    def backward(q, slopes=4096, dy=4096, lddy=40, dx=4096, dw=4096, db=4096, err=4096):
        return lib.sfnn_linear_backward(None if q is None else ctypes.byref(q), slopes, dy, lddy, dx, dw, db, 4096, 1 << 40,
                                        err, None)
    assert backward(None) == INVALID
    for kw in (dict(slopes=None), dict(slopes=4100), dict(dy=None), dict(dy=4097), dict(lddy=32), dict(dx=4104),
               dict(dw=4098), dict(db=4097), dict(err=None)):
        assert backward(linear(), **kw) == INVALID, kw
    assert lib.sfnn_linear_workspace(-1, 64, 64, 0) < 0 and lib.sfnn_linear_workspace(0, 64, 64, 1) >= 0
    assert lib.sfnn_linear_slope_bytes(3, 129, 1) == 3 * 32 and lib.sfnn_linear_slope_bytes(3, 33, 2) == 3 * 128
    assert lib.sfnn_linear_slope_bytes(3, 129, 0) == 0 and lib.sfnn_linear_slope_bytes(3, 129, 4) < 0


def test_linear_binding_refuses():
    x, w = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(40, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        sf.linear_forward(x, w)
    with pytest.raises(ValueError):
        sf.linear_forward(x, w, act="tanh")
    with pytest.raises(TypeError):
        sf.linear(x, w)
