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


# An accumulator of an fp32 result takes at most 128 steps of 16 products, each of which cuts up to 2^-23, on average
# 2^-24, off the sum so far; sums of random signs grow with the root of their length, 2/3 of the last on average, so
# that 128 2^-24 2/3 = 5.1e-6 of the result would be lost at the most.  The accumulators hold a few bits more than a
# result does: half of that for the mean over values, 128 2^-25 = 3.8e-6, is allowed.
LONG = [(28672, 7168, (1, 50, 100, 128, 200, 300, 400, 800, 1024, 1100)), (16384, 4096, (2, 160, 300, 400, 513)),
        (8192, 8192, (64, 160, 300, 800, 1024)), (65536, 1000, (3, 128, 700))]


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("K,N,tokens", LONG)
def test_long_sums_that_leave_as_fp32(K, N, tokens, dt):
    w = normal(N, K, seed=K, size=K ** -0.5, dt=dt)
    W = w.double()
    for T in tokens:
        x = normal(T, K, seed=T, dt=dt)
        want = x.double() @ W.t()
        error = sf.linear_forward(x, w, out_dtype=torch.float32)[0].double() - want
        assert error.square().mean().sqrt() <= 128 * 2.0 ** -25 * want.square().mean().sqrt(), T
    assert sf.dense_error() == 0


# silu: the exponent z log2 e is off by 1.5 roundings, which e^-z takes |z| 1.5 2^-24 of itself from; the special functions'
# 2^-22 and 2^-23 and three products' roundings: (|z| + 8) 2^-23.  Below -87.3 its 1 / (1 + e^-z) leaves the
# normal range: up to 88 2^-126 is lost.  gelu: likewise z^2 / 2 times 2.5 roundings, the polynomial's 3.7e-8 and
# its nine steps of at most twice the sum's size: (1.25 z^2 + 32) 2^-24; below -13 its e^(-z^2 / 2) leaves the range.
@pytest.mark.parametrize("T", [1, 64, 1200])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_activations_far_out(act, T):
    far = torch.cat([torch.linspace(-16, 16, 513), torch.linspace(-104, -16, 353), torch.tensor([16.0, 40, 87, 88, 89, 104, 1000, 3e4])])
    z = far.half()
    w = torch.zeros(z.numel(), 8, dtype=torch.float16)
    w[:, 0] = z
    x = torch.zeros(T, 8, dtype=torch.float16)
    x[:, 0] = 1
    y = sf.linear_forward(x.cuda(), w.cuda(), act=act, out_dtype=torch.float32)[0].double()
    z = z.double().cuda()
    # (through erfc: 1 + erf has nothing left beyond -8.3)
    want = z * 0.5 * torch.special.erfc(z * -0.5 ** 0.5) if act == "gelu" else z / (1 + torch.exp(-z))
    rel = (1.25 * z.clamp(-14, 14).square() + 32) * 2.0 ** -24 if act == "gelu" else (z.abs().clamp_max(104) + 8) * 2.0 ** -23
    tol = rel * want.abs() + (1 if act == "gelu" else 88) * 2.0 ** -126
    off = (y - want).abs() / tol
    assert (off <= 1).all(), (off.max().item(), z[off.max(0)[0].argmax()].item())
