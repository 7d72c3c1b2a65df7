"""MXFP4 quantisation against its definition (equal, value for value) and the block-scaled
product against a 64-bit one.

The product's operands are exact, so a result is off by its own rounding (eps/2) and by the
fp32 accumulation: at most K 2^-23 of the terms' magnitudes (each of fewer than K additions,
in blocks, loses at most 2^-23 of the running magnitude when an addend is cut rather than
rounded).
"""
import pathlib
import subprocess
import sys

import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu

ROOT = pathlib.Path(__file__).resolve().parent.parent

KINDS = [torch.float16, torch.bfloat16]


def values64(x):
    """The values MXFP4 holds for x [R, K], from the definition, in 64 bits."""
    R, K = x.shape
    v = x.double().view(R, K // 32, 32)
    top = v.abs().amax(2, keepdim=True)
    finite = torch.isfinite(top) & torch.isfinite(v).all(2, keepdim=True)
    e = (torch.frexp(torch.where(finite & (top > 0), top, torch.ones_like(top))).exponent - 3)
    e = torch.where(top > 0, e, -127).clamp(-127, 127).long()
    scale = ((e + 1023) << 52).view(torch.float64)
    a = v.abs() / scale
    grid = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    q = ((a / grid).round() * grid).clamp(max=6.0) * v.sign() * scale
    return torch.where(finite, q, torch.full_like(q, float("nan"))).view(R, K)


def data(R, K, dt, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(R, K, generator=g, device="cuda")
    return (x * torch.exp(spread * torch.randn(R, 1, generator=g, device="cuda"))).to(dt)


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("R,K", [(1, 32), (1, 64), (3, 96), (5, 2048), (130, 288), (257, 2080), (2, 28672)])
def test_quantize_equals_the_definition(R, K, dt):
    x = data(R, K, dt, R + K)
    if R > 1:
        x[1] = 0
    q = sf.quantize_mxfp4(x)
    got = sf.dequantize_mxfp4(q, torch.bfloat16 if dt == torch.bfloat16 else torch.float16).double()
    want = values64(x)
    # a held value has two significant bits, so it is exact in bf16; fp16 loses what lies under its smallest step
    assert torch.equal(got, want.to(dt).double())
    assert q.nbytes >= R * K // 2 + R * K // 32
    wide = torch.zeros(R, K + 5, dtype=dt, device="cuda")
    wide[:, 3: K + 3] = x
    q2 = sf.quantize_mxfp4(wide[:, 3: K + 3])
    assert torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales)


def test_every_tie_and_special_value():
    steps = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9], device="cuda")
    x = torch.zeros(8, 64, device="cuda")
    x[0, :17], x[0, 32:49] = steps, -steps
    x[1, :17], x[1, 17] = steps, 4.0
    x[2] = x[0] * 2.0 ** 100
    x[3] = x[0] * 2.0 ** -124  # scale near the lowest
    x[4, :3] = torch.tensor([1e-38, 3e-39, -1e-40])  # below the lowest scale's step and around it
    x[5, 5], x[5, 40] = float("nan"), 2.0
    x[6, 7], x[6, 41] = float("inf"), 1.0
    x[7, 33] = float("-inf")
    x = x.to(torch.bfloat16)
    got, want = sf.dequantize_mxfp4(sf.quantize_mxfp4(x)).double(), values64(x).to(torch.bfloat16).double()
    assert torch.equal(got.isnan(), want.isnan()) and got[5, :32].isnan().all() and not got[5, 32:].isnan().any()
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


SHAPES = [(1, 32, 64), (1, 1, 32), (1, 11008, 4096), (2, 33, 256), (3, 4099, 512), (4, 100, 8192), (8, 160, 288),
          (17, 257, 544), (64, 1000, 2048), (77, 4099, 96), (128, 352, 736), (129, 512, 320), (256, 256, 256),
          (300, 777, 1056), (511, 1537, 800), (1000, 2048, 2048)]


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_product(T, N, K, dt):
    x, w = data(T, K, dt, T + N), data(N, K, dt, K + 1) / K ** 0.5
    xq, wq = sf.quantize_mxfp4(x), sf.quantize_mxfp4(w)
    X, Wv = values64(x), values64(w)
    want, terms = X @ Wv.t(), X.abs() @ Wv.abs().t()
    for out in (torch.float32, dt):
        got = sf.mxfp4_matmul(xq, wq, out_dtype=out)
        assert got.shape == (T, N) and got.dtype == out
        tol = torch.finfo(out).eps / 2 * want.abs() + K * 2.0 ** -23 * terms * 1.01 + torch.finfo(out).smallest_normal
        bad = (got.double() - want).abs() > tol
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} out of bound ({out})"
        lin = sf.mxfp4_linear(x, wq, out_dtype=out)
        bad = (lin.double() - want).abs() > tol
        assert not bad.any(), f"linear: {int(bad.sum())} of {bad.numel()} out of bound ({out})"
    assert sf.dense_error() == 0


@pytest.mark.parametrize("T,N,K", [(128, 8192, 2048), (128, 4096, 1024), (100, 9400, 2048), (70, 16300, 1056)])
def test_short_products_that_fill_every_sm(T, N, K):
    """Few steps leave little shared memory to a CTA: no more of them may share an SM than
    its tensor memory holds.  Calls in a row, so that each begins while the last one ends."""
    x, w = data(T, K, torch.float16, 3), data(N, K, torch.float16, 4)
    qx, qw = sf.quantize_mxfp4(x), sf.quantize_mxfp4(w)
    want = values64(x) @ values64(w).t()
    terms = values64(x).abs() @ values64(w).abs().t()
    got = [sf.mxfp4_matmul(qx, qw, out_dtype=torch.float32) for _ in range(12)]
    assert ((got[0].double() - want).abs() <= (2.0 ** -24 + K * 2.0 ** -23) * terms).all()
    assert all(torch.equal(g, got[0]) for g in got)
    assert sf.dense_error() == 0


@pytest.mark.parametrize("T,N,K", [(129, 136, 4096), (200, 513, 4128), (300, 1000, 4640), (384, 130, 8192), (511, 264, 5120),
                                   (1000, 8, 4096), (2000, 1, 4096), (300, 11008, 288), (384, 11007, 96)])
def test_product_in_groups_of_tokens(T, N, K):
    """More than 128 tokens by 128: long K split over clusters, and tiles of one round."""
    test_product(T, N, K, torch.bfloat16)


def test_product_of_views_nan_rows_and_empty():
    x, w = data(40, 128, torch.bfloat16, 1), data(96, 128, torch.bfloat16, 2)
    wq = sf.quantize_mxfp4(w)
    want = sf.mxfp4_linear(x, wq)
    assert torch.equal(sf.mxfp4_linear(x.view(2, 20, 128), wq).view(40, 96), want)
    wide = torch.randn(40, 131, device="cuda").to(torch.bfloat16)
    wide[:, 1:129] = x
    assert torch.equal(sf.mxfp4_linear(wide[:, 1:129], wq), want)
    for rows in (1, 2, 40):
        x2 = x[:rows].clone()
        x2[rows - 1, 70] = float("nan")
        got = sf.mxfp4_linear(x2, wq)
        assert got[rows - 1].isnan().all() and torch.equal(got[:rows - 1], sf.mxfp4_linear(x, wq)[:rows - 1]) or rows < 3
    assert sf.mxfp4_linear(x[:0], wq).shape == (0, 96)
    w2 = w.clone()
    w2[5, 3] = float("inf")
    got = sf.mxfp4_linear(x, sf.quantize_mxfp4(w2))
    keep = [i for i in range(96) if i != 5]
    assert got[:, 5].isnan().all() and torch.equal(got[:, keep], want[:, keep])


def test_large_and_small_scales():
    x = data(6, 256, torch.bfloat16, 3)
    for kx, kw in ((2.0 ** 60, 2.0 ** 50), (2.0 ** -60, 2.0 ** -50), (2.0 ** 100, 2.0 ** -100)):
        w = data(64, 256, torch.bfloat16, 4)
        for rows in (1, 6):
            xs, ws = (x[:rows].float() * kx).to(torch.bfloat16), (w.float() * kw).to(torch.bfloat16)
            got = sf.mxfp4_linear(xs, sf.quantize_mxfp4(ws), out_dtype=torch.float32)
            base = sf.mxfp4_linear(x[:rows], sf.quantize_mxfp4(w), out_dtype=torch.float32)
            assert torch.equal(got.double(), base.double() * (kx * kw))  # powers of two move nothing else


def test_graph_and_streams():
    x, w = data(5, 512, torch.float16, 5), data(300, 512, torch.float16, 6)
    wq = sf.quantize_mxfp4(w)
    xs = [x, data(200, 512, torch.float16, 7), x[:1].clone()]
    want = [sf.mxfp4_linear(a, wq) for a in xs]
    graphs = []
    for a in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = sf.mxfp4_linear(a, wq)
        graphs.append((g, y))
    for k in (0, 1, 2, 1, 0, 2):
        graphs[k][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[k][1], want[k])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [(k, sf.mxfp4_linear(xs[k], wq, stream=streams[k])) for _ in range(5) for k in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k, y in outs)
    assert sf.dense_error() == 0


def test_outputs_beyond_32_bits():
    T, N, K = 70001, 32768, 64
    x, w = data(T, K, torch.bfloat16, 11), data(N, K, torch.bfloat16, 12)
    wq = sf.quantize_mxfp4(w)
    y = sf.mxfp4_linear(x, wq)
    rows = torch.tensor([0, 255, 40000, T - 130, T - 1], device="cuda")
    want = values64(x[rows]) @ values64(w).t()
    # half a step of bf16 is 2^-8 of the value (165.5 may go to 166: its neighbours are 1 apart)
    tol = torch.finfo(torch.bfloat16).eps / 2 * want.abs() + K * 2.0 ** -23 * (values64(x[rows]).abs() @ values64(w).abs().t()) + 1e-30
    assert ((y[rows].double() - want).abs() <= tol).all()
    assert sf.dense_error() == 0


def test_workspace_and_error_word_are_apart_in_a_new_process():
    """The process's first dense call allocates the error word while the call's workspace lives."""
    code = """
import torch
import activation_sparse_ffn_threshold_b200 as sf
g = torch.Generator(device="cuda").manual_seed(1)
w = sf.quantize_mxfp4(torch.randn(64, 256, device="cuda", generator=g).half())
x = torch.randn(8, 256, device="cuda", generator=g).half()
for _ in range(3):
    sf.mxfp4_linear(x, w)
assert sf.dense_error() == 0, "the error word was written to"
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
