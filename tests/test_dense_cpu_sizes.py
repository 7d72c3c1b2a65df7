"""Sizes near and beyond the end of 32 bits, refused without a GPU."""
import warnings

import pytest
import torch

from activation_sparse_ffn_threshold_b200 import dense


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
