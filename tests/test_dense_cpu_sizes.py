"""Sizes near and beyond the end of 32 bits and addresses off their alignment, refused without a GPU."""
import ctypes
import warnings

import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf
from activation_sparse_ffn_threshold_b200 import dense
from test_dense_cpu import INVALID, UNSUPPORTED, desc, forward, saved_of


def test_binding_refuses_sizes_that_32_bits_do_not_hold():
    """The C entry points take 32-bit sizes, and ctypes cuts larger ones without a word."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")  # (a fake tensor has no address)
        flat = torch.empty(2 ** 32 + 64, dtype=torch.float16, device="cuda")
        tall = torch.empty(2 ** 32 + 1, 8, dtype=torch.float16, device="cuda")
        for t in (flat, flat.view(1, -1), tall, tall.view(2 ** 32 + 1, 1, 8), tall[:, :4]):
            with pytest.raises(ValueError, match="32"):
                dense._rows(t, "x")
        edge = torch.empty(2 ** 31 - 1, 8, dtype=torch.float16, device="cuda")
        assert dense._rows(edge, "x")[1:] == (2 ** 31 - 1, 8, 8)


def test_act8_refuses_widths_near_the_end_of_32_bits():
    lib = sf.load_library()
    for cols in (65535 * 2048 + 1, 2 ** 31 - 2048, 2 ** 31 - 64, 2 ** 31 - 1):  # more than a launch's grid covers
        args = (4096, cols, 1, cols, sf.F16, 0)
        assert lib.sfnn_act8_quantize(*args, 4096, 2 ** 31, 4096, 2 ** 25, None) == UNSUPPORTED, cols
        assert lib.sfnn_act8_restore(4096, 2 ** 31, 4096, 2 ** 25, 1, cols, 0, sf.F16, 4096, cols, None) == UNSUPPORTED, cols


def test_addresses_off_their_types_alignment_are_refused():
    """A kernel that loads or stores there would fault."""
    lib = sf.load_library()
    assert forward(desc(b=4097)) == INVALID and forward(desc(), err=4098) == INVALID
    for kind, name in ((1, "r_scales"), (1, "u_scales"), (2, "r_scales"), (2, "u_scales"), (2, "x_scales")):
        s = saved_of(kind=kind)
        setattr(s, name, 4098)
        assert forward(desc(), saved=s) == INVALID, name

    def back(s=None, db=4096, err=4096):
        q, s = desc(), s or saved_of()
        return lib.sfnn_gated_backward(ctypes.byref(q), 4096, 64, ctypes.byref(s), 4096, 4096, 4096, 4096, db, 4096, 1 << 40,
                                       err, None)
    s = saved_of()
    s.u_scales = 4098
    assert back(s) == INVALID and back(db=4097) == INVALID and back(err=4098) == INVALID
    assert lib.sfnn_mxfp4_product(4096, 4096, 4, 4096, 4096, 8, 64, 4096, 8, sf.F32, 4098, None) == INVALID
    assert lib.sfnn_mxfp4_linear(4096, 64, 16, sf.F16, 4096, 4096, 8, 64, 4096, 8, sf.F16, 4096, 1 << 30, 4098, None) == INVALID
