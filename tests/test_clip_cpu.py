"""The clipping's refusals of overlapping memory in C, which need no GPU."""
import ctypes

import pytest

import activation_sparse_ffn_threshold_b200 as sf

INVALID = sf.STATUS_CODES["SFNN_ERR_INVALID_ARG"]
A, B, C, D = (1 << 40) + 4096, (2 << 40), (3 << 40), (4 << 40)  # far apart; nothing there is touched: the call is refused


def clip(rows, norm, ws):
    lib = sf.load_library()
    flat = [v for r in rows for v in r]
    return lib.sfnn_clip_grad_norm((ctypes.c_int64 * len(flat))(*flat), len(rows), 1.0, 1.0, 1e-6, norm, ws, 1 << 30, None)


@pytest.mark.parametrize("at", [A, A + 4, A + 1996, B, B + 1996])
def test_a_norm_inside_a_gradient_or_an_output(at):
    assert clip([(A, B, 1000, sf.F16)], at, D) == INVALID


@pytest.mark.parametrize("at", [A, A + 1992, A - 8, B, B + 1992, B - 56])
def test_a_workspace_over_a_gradient_or_an_output(at):
    assert clip([(C, C, 8, sf.F32), (A, B, 1000, sf.F16)], D, at) == INVALID


@pytest.mark.parametrize("at", [D, D + 4, D + 60])
def test_a_norm_inside_the_workspace(at):
    assert clip([(A, B, 1000, sf.F16)], at, D) == INVALID
