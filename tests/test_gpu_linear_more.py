"""The linear layer where other tests of it do not go: products at the same time, long sums that leave as fp32,
activations far out, transforms of autograd."""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu


def normal(*shape, seed, size=1.0, dt=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * size).to(dt)


# K split over clusters of 2 to 8, the sums exchanged in memory of their own and in the stages'.
SPLIT = [(1, 4096, 1000), (8, 4096, 4096), (32, 4096, 4096), (50, 16384, 4096), (100, 8192, 2048), (250, 8192, 3500),
         (16, 28672, 515), (512, 4096, 1024)]


def test_split_products_on_two_streams_at_once():
    """Clusters of two products share the SMs, and each gives what it gives alone."""
    for i, first in enumerate(SPLIT):
        second = SPLIT[(3 * i + 1) % len(SPLIT)]
        sets = [(normal(T, K, seed=i, dt=torch.float16), normal(N, K, seed=i + 9, size=K ** -0.5, dt=torch.float16),
                 normal(N, seed=i + 18, dt=torch.float16)) for T, K, N in (first, second)]
        alone = [sf.linear_forward(x, w, b, "gelu")[0] for x, w, b in sets]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in sets]
        out = [[], []]
        for _ in range(20):
            for j, (s, (x, w, b)) in enumerate(zip(streams, sets)):
                out[j].append(sf.linear_forward(x, w, b, "gelu", stream=s)[0])
        torch.cuda.synchronize()
        for got, want in zip(out, alone):
            assert all(torch.equal(y, want) for y in got)
    assert sf.dense_error() == 0
