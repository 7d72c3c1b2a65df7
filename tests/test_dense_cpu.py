"""Refusals of the dense operators, which need no GPU: the C entry points return a status
and launch nothing, the binding raises."""
import ctypes

import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf
from activation_sparse_ffn_threshold_b200 import dense

INVALID, UNSUPPORTED = sf.STATUS_CODES["SFNN_ERR_INVALID_ARG"], sf.STATUS_CODES["SFNN_ERR_UNSUPPORTED"]


def desc(T=4, d=64, n=128, dtype=sf.F16, layout=0, **kw):
    q = dense._GatedDesc(T, d, n, dtype, layout, 0, 4096, d, 4096, d, 4096, d, 4096, n if layout == 0 else d, None)
    for k, v in kw.items():
        setattr(q, k, v)
    return q


def forward(q, y=4096, ldy=None, y_dtype=None, saved=None, ws=4096, ws_bytes=1 << 40, err=4096):
    return sf.load_library().sfnn_gated_forward(ctypes.byref(q), y, q.d if ldy is None else ldy,
                                                q.dtype if y_dtype is None else y_dtype,
                                                None if saved is None else ctypes.byref(saved), ws, ws_bytes, err, None)


def saved_of(T=4, d=64, n=128, kind=1):
    s = dense._GatedSaved(kind, 0, 4096, 4096, -(-n // 64) * 64, 4096, 4096, -(-n // 64), 4096,
                          -(-d // 64) * 64, 4096, -(-d // 64))
    return s


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(n=0), INVALID), (dict(dtype=7), INVALID),
    (dict(dtype=sf.F32), UNSUPPORTED), (dict(d=60), UNSUPPORTED), (dict(n=132), UNSUPPORTED),
    (dict(d=(1 << 20) + 8), UNSUPPORTED), (dict(n=(1 << 20) + 8), UNSUPPORTED), (dict(T=(1 << 24) + 1), UNSUPPORTED),
    (dict(layout=2), INVALID), (dict(x=None), INVALID), (dict(x=4104), INVALID), (dict(ldx=60), INVALID),
    (dict(ldx=68), INVALID), (dict(w_gate=None), INVALID), (dict(w_up=8), INVALID), (dict(ld_up=66), INVALID),
    (dict(w_down=None), INVALID), (dict(ld_down=120), INVALID)])
def test_forward_refuses_bad_descriptors(kw, want):
    assert forward(desc(**kw)) == want


def test_forward_refuses_bad_buffers():
    q = desc()
    need = sf.load_library().sfnn_gated_workspace(4, 64, 128, 0)
    assert need >= 4 * 128 * 2
    assert forward(q, y=None) == INVALID and forward(q, y=4100) == INVALID and forward(q, ldy=56) == INVALID
    assert forward(q, y_dtype=sf.BF16) == INVALID and forward(q, ws=None) == INVALID
    assert forward(q, ws_bytes=need - 1) == INVALID and forward(q, err=None) == INVALID
    bad = saved_of()
    bad.ld = 120
    assert forward(q, saved=bad) == INVALID
    bad = saved_of(kind=2)
    bad.x_scales = None
    assert forward(q, saved=bad) == INVALID
    bad = saved_of(kind=2)
    bad.ld_x = 56
    assert forward(q, saved=bad) == INVALID
    bad = saved_of(kind=5)
    assert forward(q, saved=bad) == INVALID
    assert sf.load_library().sfnn_gated_forward(None, 4096, 64, 1, None, 4096, 1 << 30, 4096, None) == INVALID
    assert forward(desc(T=0)) == 0  # no token: nothing to do


def test_backward_refuses():
    lib = sf.load_library()

    def back(q, s, dy=4096, lddy=64, ws=4096, nbytes=1 << 40, dx=4096):
        return lib.sfnn_gated_backward(None if q is None else ctypes.byref(q), dy, lddy,
                                       None if s is None else ctypes.byref(s), dx, 4096, 4096, 4096, 4096, ws, nbytes,
                                       4096, None)
    assert back(None, saved_of()) == INVALID and back(desc(), None) == INVALID
    assert back(desc(), saved_of(kind=0)) == INVALID
    assert back(desc(layout=1), saved_of()) == UNSUPPORTED
    assert back(desc(), saved_of(), dy=None) == INVALID and back(desc(), saved_of(), lddy=32) == INVALID
    assert back(desc(), saved_of(), nbytes=1024) == INVALID and back(desc(), saved_of(), dx=4098) == INVALID
    assert lib.sfnn_gated_workspace(-1, 64, 64, 0) < 0
    assert lib.sfnn_forward_prompt(None, 4096, 1, 4096, 4096, 1 << 30, None) == INVALID


def test_act8_refuses():
    lib = sf.load_library()

    def quant(T=2, cols=100, ldx=100, dtype=sf.F16, x=4096, codes=4096, ldq=128, scales=4096, lds=2):
        return lib.sfnn_act8_quantize(x, ldx, T, cols, dtype, 0, codes, ldq, scales, lds, None)
    for kw in (dict(T=-1), dict(cols=0), dict(ldx=99), dict(dtype=sf.F32), dict(x=None), dict(codes=None),
               dict(codes=4100), dict(ldq=112), dict(ldq=130), dict(scales=None), dict(scales=4098), dict(lds=1),
               dict(x=4097)):
        assert quant(**kw) == INVALID, kw
    assert quant(T=0) == 0
    assert lib.sfnn_act8_restore(4096, 128, 4096, 2, 2, 100, 0, sf.I8, 4096, 100, None) == INVALID


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.float16)
    w, wd = torch.zeros(128, 64, dtype=torch.float16), torch.zeros(64, 128, dtype=torch.float16)
    with pytest.raises(TypeError):
        sf.gated_ffn_forward(x, w, w, wd)
    with pytest.raises(ValueError):
        sf.gated_ffn_forward(x, w, w, wd, save="int8")
    with pytest.raises(ValueError):
        sf.gated_ffn(x, w, w, wd, checkpoint=None)
    with pytest.raises(TypeError):
        sf.quantize_act8(x)
    with pytest.raises(TypeError):
        sf.quantize_act8(x.float())


def test_mxfp4_refuses():
    lib = sf.load_library()
    assert lib.sfnn_mxfp4_scale_bytes(1, 32) == 2 * 2 * 512 and lib.sfnn_mxfp4_scale_bytes(257, 288) == 4 * 4 * 512
    assert lib.sfnn_mxfp4_scale_bytes(-1, 32) < 0 and lib.sfnn_mxfp4_linear_workspace(1, 0) < 0

    def quant(x=4096, ldx=64, rows=2, K=64, dtype=sf.F16, codes=4096, scales=4096):
        return lib.sfnn_mxfp4_quantize(x, ldx, rows, K, dtype, codes, scales, None)
    for kw, want in ((dict(x=None), INVALID), (dict(ldx=63), INVALID), (dict(rows=-1), INVALID), (dict(K=0), INVALID),
                     (dict(K=48, ldx=48), UNSUPPORTED), (dict(dtype=sf.F32), INVALID), (dict(codes=4104), INVALID),
                     (dict(scales=None), INVALID), (dict(K=(1 << 20) + 32, ldx=1 << 21), UNSUPPORTED),
                     (dict(rows=(1 << 24) + 1), UNSUPPORTED)):
        assert quant(**kw) == want, kw
    assert quant(rows=0) == 0
    assert lib.sfnn_mxfp4_restore(4096, 4096, 2, 64, sf.I4, 4096, 64, None) == INVALID

    def prod(xc=4096, T=4, wc=4096, N=8, K=64, y=4096, ldy=8, dt=sf.F32, err=4096):
        return lib.sfnn_mxfp4_product(xc, 4096, T, wc, 4096, N, K, y, ldy, dt, err, None)
    for kw in (dict(xc=None), dict(T=-1), dict(wc=8), dict(N=0), dict(y=None), dict(ldy=7), dict(dt=sf.I8),
               dict(err=None), dict(y=4097)):
        assert prod(**kw) == INVALID, kw
    assert prod(K=40) == UNSUPPORTED and prod(T=0) == 0

    def linear(ws=4096, nbytes=1 << 30, x=4096, ldx=64):
        return lib.sfnn_mxfp4_linear(x, ldx, 16, sf.F16, 4096, 4096, 8, 64, 4096, 8, sf.F16, ws, nbytes, 4096, None)
    assert linear(ws=None) == INVALID and linear(nbytes=8) == INVALID and linear(x=None) == INVALID
    assert linear(ldx=32) == INVALID
    with pytest.raises(TypeError):
        sf.quantize_mxfp4(torch.zeros(2, 64, dtype=torch.float16))
    with pytest.raises(TypeError):
        sf.mxfp4_linear(torch.zeros(2, 64, dtype=torch.float16), None)


def test_workspace_of_no_tokens():
    lib = sf.load_library()
    assert lib.sfnn_gated_workspace(0, 64, 128, 0) >= 0 and lib.sfnn_gated_workspace(0, 64, 128, 1) >= 0
