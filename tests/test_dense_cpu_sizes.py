"""Sizes near and beyond the end of 32 bits, refused without a GPU."""
import warnings

import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf
from activation_sparse_ffn_threshold_b200 import dense

UNSUPPORTED = sf.STATUS_CODES["SFNN_ERR_UNSUPPORTED"]


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
