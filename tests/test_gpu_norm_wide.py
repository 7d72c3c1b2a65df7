"""Norms of many rows 4097 to 8192 wide, where an SM's shared memory holds few rows of an fp32 stream: one
group of threads, two stages or one, with and without vectors."""
import pytest
import torch

from test_gpu_block import check

pytestmark = pytest.mark.gpu

KINDS = [torch.float16, torch.bfloat16]


@pytest.mark.parametrize("d", [4097, 5120, 6656, 7000, 8184, 8191, 8192])
@pytest.mark.parametrize("pre,post,gate", [("rms", "rms", "vec"), ("layer", "none", None), ("layer", "rms", "token"),
                                           ("rms", "layer", None)])
def test_an_fp32_stream(d, pre, post, gate):
    for i, T in enumerate((149, 601)):
        check(T, d, KINDS[(d + i) % 2], A=[1.0, 0.75][i], C=[1.0, -0.5][i], seed=d + i, pre=pre, post=post, gate=gate,
              bias=pre == "layer", x32=True, z32=i == 1)
