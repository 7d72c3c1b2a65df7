"""The linear layer with its epilogue and its gradients against plain 64-bit computations.

Tolerances.  A result is rounded once to its type (half a step: eps / 2 of the value).  Its sum of K
products in 32 bits is off by at most K 2^-23 of the terms' magnitudes; an activation passes that on
with a slope of at most 1.13, and its own evaluation adds (|z| + 8) 2^-23 of the value (an exponent's
rounding grows with |z|; the normal integral is good to 5 ulp).  dZ carries act', held to 2^-16 (a
ReLU's exactly) and off by 0.8 of z's error, and its rounding, eps / 2, for the products."""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu

KINDS = [torch.float16, torch.bfloat16]
ACTS = ["none", "relu", "gelu", "silu"]


def make(T, K, N, dt, act, res=None, bias=True, seed=0, pad=0, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = torch.zeros(T, K + pad, device="cuda", dtype=dt)
    # on grids, so that sums are exact in fp32 and a ReLU's side is certain
    x[:, :K] = ((r(T, K) * 16).round() / 16).clamp(-4, 4)
    unit = 2.0 ** round(torch.log2(torch.tensor(0.25 / K ** 0.5)).item())
    w = ((r(N, K) * 4).round().clamp(-16, 16) * unit).to(dt)
    b = ((r(N) * 8).round() / 32).to(dt) if bias else None

    def values(size=1.0):  # rows at any alignment
        t = torch.float32 if res == "f32" else dt
        buf = torch.full((T * (N + pad) + off,), 7.0, device="cuda", dtype=t)
        v = buf[off:].view(T, N + pad)[:, :N]
        v.copy_(r(T, N) * size)
        return v
    return x[:, :K], w, b, values() if res else None, values


def activation(z, act):
    z = z.detach().requires_grad_()
    y = {"none": lambda: z * 1, "relu": lambda: z.clamp_min(0) * 1, "silu": lambda: z * torch.sigmoid(z),
         "gelu": lambda: z * torch.special.ndtr(z)}[act]()
    (d,) = torch.autograd.grad(y.sum(), z)
    if act == "relu":
        d = (z > 0).double()
    return y.detach(), d


def near(got, want, extra):
    info = torch.finfo(got.dtype)
    tol = info.eps / 2 * want.abs() + extra + info.smallest_normal * info.eps
    bad = ~((got.double() - want).abs() <= 1.001 * tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} out of bound, worst " \
                          f"{((got.double() - want).abs() / tol).max().item():.2f} times"


def forward64(x, w, b, act, res):
    X, W = x.double(), w.double()
    z, za = X @ W.t(), X.abs() @ W.abs().t()
    if b is not None:
        z, za = z + b.double(), za + b.double().abs()
    y, slope = activation(z, act)
    ez = x.shape[-1] * 2.0 ** -23 * za
    if act == "relu":
        ez = ez * 0  # exact
    extra = 1.13 * ez + (0 if act in ("none", "relu") else (z.abs() + 8) * 2.0 ** -23 * y.abs())
    if res is not None:
        y = y + res.double()
        extra = extra + 2.0 ** -24 * (y.abs() + res.double().abs())
    return y, extra, z, slope, ez


def check(T, K, N, dt, act, res=None, save=True, **kw):
    x, w, b, r, values = make(T, K, N, dt, act, res, **kw)
    want, extra, z, slope, ez = forward64(x, w, b, act, r)
    for keep in (False, True)[:1 + save]:
        y, saved = sf.linear_forward(x, w, b, act, r, save=keep)
        assert y.dtype == (r.dtype if r is not None else dt) and y.shape == (T, N)
        near(y, want, extra)
    if not save:
        return
    dy = values(0.5)
    if res is None:
        dy = dy.to(dt)
    got = sf.linear_backward(dy, saved, w)
    D = dy.double()
    dz = D * slope
    # dZ's error: its rounding, act's
    smooth = act in ("gelu", "silu")
    info = torch.finfo(dt)
    as_is = act == "none" and res != "f32"
    edz = (0 if as_is else info.eps / 2 * dz.abs() + info.smallest_normal * info.eps) + \
        (D.abs() * (2.0 ** -16 + 2.0 ** -20 + 0.8 * ez) if smooth else 0 * dz)
    X, W = x.double(), w.double()
    near(got[0], dz @ W, edz @ W.abs() + N * 2.0 ** -23 * (dz.abs() @ W.abs()))
    near(got[1], dz.t() @ X, edz.t() @ X.abs() + T * 2.0 ** -23 * (dz.abs().t() @ X.abs()))
    if b is None:
        assert got[2] is None
    else:  # before dZ's rounding
        e = (D.abs() * (2.0 ** -16 + 2.0 ** -20 + 0.8 * ez) if smooth else 0 * dz).sum(0)
        near(got[2], dz.sum(0), e + T * 2.0 ** -23 * dz.abs().sum(0))
    again = sf.linear_backward(dy, saved, w)
    assert all(u is v is None or torch.equal(u, v) for u, v in zip(got, again))
    for i in range(3):  # one at a time
        need = [j == i for j in range(3)]
        one = sf.linear_backward(dy, saved, w, need=need)
        assert all((t is not None) == (j == i and got[j] is not None) for j, t in enumerate(one))
        if got[i] is not None:
            near(one[i], got[i].double(), (info.eps + T * 2.0 ** -22) * got[i].double().abs() + 2.0 ** -20) if i == 2 else None
            assert i == 2 or torch.equal(one[i], got[i])
    assert sf.dense_error() == 0


SHAPES = [(1, 8, 1), (1, 512, 2048), (2, 64, 64), (3, 72, 33), (5, 40, 130), (31, 136, 1000), (77, 1000, 515),
          (128, 64, 257), (129, 200, 264), (257, 520, 512), (300, 1000, 2047)]


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_sizes(T, K, N, act, dt):
    i = T + K + N + ACTS.index(act)
    check(T, K, N, dt, act, res=[None, "same", "f32"][i % 3], bias=i % 4 != 0, seed=i, pad=8 * (i % 2))


@pytest.mark.parametrize("T,K,N", [(1, 4096, 16384), (4, 16384, 4096), (50, 7168, 1000), (128, 9504, 2048), (16, 280, 20311),
                                   (2100, 1104, 520), (700, 264, 2504), (64, 8192, 96), (130, 8200, 101), (2500, 64, 40)])
def test_long_ones(T, K, N):
    act = ACTS[(T + K) % 4]
    check(T, K, N, KINDS[N % 2], act, res=["f32", None, "same"][T % 3], seed=T)


@pytest.mark.parametrize("res", ["same", "f32"])
@pytest.mark.parametrize("T", [4, 200])
@pytest.mark.parametrize("pad,off", [(8, 8), (8, 0), (3, 0), (0, 1), (2, 2)])
def test_alignments_of_the_output_side(pad, off, T, res):
    x, w, b, r, values = make(T, 136, 264, torch.bfloat16, "silu", res, seed=T)
    want, extra, z, slope, _ = forward64(x, w, b, "silu", r)
    _, saved = sf.linear_forward(x, w, b, "silu", r, save=True)
    plain = sf.linear_forward(x, w, b, "silu", r)[0]
    near(plain, want, extra)
    buf = torch.full((T * (264 + pad) + off,), 5.0, device="cuda", dtype=r.dtype)
    view = buf[off:].view(T, 264 + pad)[:, :264]
    view.copy_(r)
    y, _ = sf.linear_forward(x, w, b, "silu", view)  # a residual anywhere
    assert torch.equal(y, plain)
    y, _ = sf.linear_forward(x, w, b, "silu", view, out=view)  # in place
    assert y is view and torch.equal(y, plain)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest[off:].view(T, 264 + pad)[:, :264] = False
    assert (buf[rest] == 5).all()
    dy = values()
    view.copy_(dy)
    for u, v in zip(sf.linear_backward(view, saved, w), sf.linear_backward(dy.contiguous(), saved, w)):
        assert torch.equal(u, v)
    assert sf.dense_error() == 0


def test_out_dtype_leading_dimensions_and_no_tokens():
    x, w, b, _, _ = make(12, 64, 40, torch.float16, "none")
    y = sf.linear_forward(x, w, b)[0]
    y3, saved = sf.linear_forward(x.view(3, 4, 64), w, b, out_dtype=torch.float32, save=True)
    assert y3.shape == (3, 4, 40) and y3.dtype == torch.float32 and torch.equal(y3.half().view(12, 40), y)
    g = sf.linear_backward(y3, saved, w)
    assert g[0].shape == (3, 4, 64)
    y1 = sf.linear_forward(x[0], w, b)[0]
    assert y1.shape == (40,)
    y0, saved = sf.linear_forward(x[:0], w, b, "gelu", save=True)
    g = sf.linear_backward(y0, saved, w)
    assert y0.shape == (0, 40) and g[0].shape == (0, 64) and (g[1] == 0).all() and (g[2] == 0).all()
    assert sf.dense_error() == 0


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_values_at_the_ends_of_the_range(act, T):
    """Saturated activations, infinities and NaNs: the limits of the formulas, a NaN stays one."""
    x, w, b, _, _ = make(T, 64, 72, torch.bfloat16, act)
    b[:8] = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), float("nan"), 100.0, -100.0, 50.0])
    y, saved = sf.linear_forward(x, w, b, act, save=True)
    assert torch.equal(sf.linear_forward(x, w, b, act)[0].isnan(), y.isnan())
    assert (y[:, 0] == b[0]).all() and (y[:, 2] == float("inf")).all() and y[:, 4].isnan().all()
    assert (y[:, [1, 3, 6]].abs() < 1e-30).all() and torch.isfinite(y[:, 5:]).all()
    dy = torch.ones_like(y)
    dx, dw, db = sf.linear_backward(dy, saved, w)
    assert torch.equal(db[[0, 1, 2, 3]], torch.tensor([T, 0.0, T, 0.0], device="cuda").bfloat16())
    assert db[4] == T if act == "relu" else (db[4].isnan() and dx.isnan().all() and dw[4].isnan().all())
    assert torch.isfinite(db[5:]).all() and torch.isfinite(dw[5:]).all()
    assert sf.dense_error() == 0


@pytest.mark.parametrize("act", ACTS)
def test_autograd_and_differences(act):
    x, w, b, r, values = make(37, 64, 56, torch.bfloat16, act, "f32", seed=5)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, r)]
    y = sf.linear(leaves[0], leaves[1], leaves[2], act, leaves[3])
    y0, saved = sf.linear_forward(x, w, b, act, r, save=True)
    assert torch.equal(y, y0)
    dy = values()
    got = torch.autograd.grad(y, leaves, dy, retain_graph=True)
    want = sf.linear_backward(dy, saved, w)
    for u, v in zip(got, want + (dy,)):
        assert torch.equal(u, v)
    # along random directions against central differences in 64 bits (a ReLU's z lies on a grid: no step
    # of 1e-7 crosses its border)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i, t in enumerate((x, w, b)):
        v = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(s):
            a = [x.double(), w.double(), b.double()]
            a[i] = a[i] + s * v
            return (activation(a[0] @ a[1].t() + a[2], act)[0] * dy.double()).sum()
        at_border = act == "relu" and bool((x.double() @ w.double().t() + b.double() == 0).any())
        if at_border:
            continue
        slope = (loss(1e-7) - loss(-1e-7)) / 2e-7
        a = (got[i].double() * v).sum()
        # roundings of dZ and of the result, 2^-9 each, on every term; differences: 2^-53 / 1e-7 of the loss's terms
        terms = (dy.double().abs() * 1.13) @ w.double().abs() if i == 0 else None
        terms = terms if i == 0 else (dy.double().abs() * 1.13).t() @ x.double().abs() if i == 1 else dy.double().abs().sum(0) * 1.13
        assert abs(a - slope) <= (2.0 ** -8 * terms * v.abs()).sum() + 1e-5 * (1 + abs(slope))
    (gx,) = torch.autograd.grad(y.sum(), leaves[0])  # an expanded gradient
    assert torch.equal(gx, sf.linear_backward(torch.ones_like(y), saved, w)[0])
    with pytest.raises(RuntimeError):
        (gx,) = torch.autograd.grad(sf.linear(leaves[0], w, b, act).sum(), leaves[0], create_graph=True)
        gx.sum().backward()


@pytest.mark.parametrize("T", [3, 200])
def test_graphs_and_streams(T):
    x, w, b, r, values = make(T, 264, 520, torch.float16, "gelu", "same")
    dy = values()

    def step():
        y, saved = sf.linear_forward(x, w, b, "gelu", r, save=True)
        return (y, sf.linear_forward(x, w, b, "relu")[0]) + sf.linear_backward(dy, saved, w)
    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, saved = sf.linear_forward(x, w, b, "gelu", r, save=True, stream=side)
    g = sf.linear_backward(dy, saved, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, first[0]) and all(torch.equal(u, v) for u, v in zip(g, first[2:]))
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(T, 264, generator=gen, device="cuda"))
        w.mul_(0.5)
        for graph in graphs:
            graph.replay()
        for out in outs:
            assert all(torch.equal(u, v) for u, v in zip(out, step()))
    assert sf.dense_error() == 0


# Few tokens: 1, 2, 4 and 8 CTAs to a tile's K, one and two halves of 128 weight rows, one tile of tokens and
# several, one round of tiles and more, the exchange in memory of its own and in the stages', ragged ends.
FEW = [(3, 8, 3977), (13, 48, 1434), (85, 568, 1), (831, 24, 7510), (3, 96, 19009), (327, 8, 18255), (275, 304, 27645),
       (80, 16, 10328), (310, 8, 25612), (196, 1776, 5647), (8, 624, 1961), (321, 1576, 3157), (852, 1384, 1664),
       (35, 624, 1246), (83, 2208, 10924), (269, 2016, 6115), (104, 1840, 2083), (193, 1208, 1603), (971, 816, 40),
       (212, 520, 3), (35, 2856, 5591), (269, 3512, 3363), (167, 1704, 2414), (65, 3968, 937), (1, 4600, 101),
       (144, 3656, 679), (569, 3880, 6), (1, 6328, 2095), (264, 9144, 1697), (187, 7128, 957), (1024, 1024, 1000)]


@pytest.mark.parametrize("T,K,N", FEW)
def test_few_tokens(T, K, N):
    for j in range(4):
        i = T + K + N + j
        check(T, K, N, KINDS[j % 2], ACTS[i % 4], res=["f32", None, "same"][i % 3], bias=i % 5 != 0, seed=i)


def test_few_tokens_leave_the_rows_beside_them():
    """Rows past the last token and columns past the last are as they were, residual in place."""
    for T, K, N in [(9, 640, 131), (300, 1024, 515), (33, 4096, 1030)]:
        x, w, b, _, _ = make(T, K, N, torch.float16, "relu", seed=T)
        for dt in (torch.float16, torch.float32):
            frame = torch.full((T + 3, N + 5), 3.0, device="cuda", dtype=dt)
            y = frame[1:T + 1, 2:N + 2]
            want, extra, *_ = forward64(x, w, b, "relu", y)
            sf.linear_forward(x, w, b, "relu", y, out=y)
            near(y, want, extra)
            edge = frame.clone()
            edge[1:T + 1, 2:N + 2] = 3.0
            assert torch.equal(edge, torch.full_like(edge, 3.0))


def test_few_tokens_of_products_in_turn():
    """A product's launch does not depend on those before it in the process, short K and long."""
    for T, K, N in [(5, 64, 77), (250, 8192, 3500), (6, 160, 3404), (250, 28672, 3800), (2, 1688, 597), (250, 12448, 4487)]:
        x, w, b, _, _ = make(T, K, N, torch.bfloat16, "none", seed=K)
        want, extra, *_ = forward64(x, w, b, "none", None)
        near(sf.linear_forward(x, w, b)[0], want, extra)


def test_out_that_shares_memory():
    x = torch.randn(6, 64, device="cuda").half()
    w = torch.randn(64, 64, device="cuda").half()
    b = torch.randn(64, device="cuda").half()
    buf = torch.zeros(7, 192, device="cuda", dtype=torch.float16)
    left, right, late = buf[:6, :64], buf[:6, 64:128], buf[:6, 72:136]
    left.copy_(x)
    want = sf.linear_forward(x, w, b)[0]
    assert torch.equal(sf.linear_forward(left, w, b, out=right)[0], want)  # side by side
    for kw in (dict(x=x, out=x), dict(x=left, out=left), dict(x=left, out=buf[:6, 8:72]), dict(x=x, w=w, out=w[:6]),
               dict(x=x[:1], b=b, out=b[None]), dict(x=x, residual=right, out=late), dict(x=x, residual=right, out=buf[1:, 64:128]),
               dict(x=left, out=buf.view(-1)[:6 * 64].view(6, 64))):
        kw = dict(w=w, b=None) | kw
        with pytest.raises(ValueError, match="overlap"):
            sf.linear_forward(**kw)
    right.copy_(x)
    assert torch.equal(sf.linear_forward(x, w, b, residual=right, out=right)[0], sf.linear_forward(x, w, b, residual=x)[0])


# Gradients' products of enough rows for tiles of 512: rows, columns and K that fill none of them.
@pytest.mark.parametrize("T,K,N", [(2500, 1000, 2600), (2305, 1160, 2311), (4100, 600, 4503), (2049, 1288, 5000)])
@pytest.mark.parametrize("dt", KINDS)
def test_gradients_of_many_rows(T, K, N, dt):
    check(T, K, N, dt, "relu", res=None, seed=T)
    check(T, K, N, dt, "silu", res="f32", bias=False, seed=N)


@pytest.mark.parametrize("T,K,N", [(1, 64, 1 << 20), (300, 64, 200003), (2, 1 << 20, 24), (1030, 8, 3), (1024, 64, 70001)])
def test_ends_of_the_range(T, K, N):
    check(T, K, N, KINDS[T % 2], "relu", res=[None, "f32"][T % 2], seed=T, save=T * N < 1 << 25)


def test_first_calls_inside_a_capture():
    """Only the error word lies on the device: kernels' limits and clusters are looked up while capturing."""
    import subprocess
    import sys
    code = """
import torch
import activation_sparse_ffn_threshold_b200 as sf
x = torch.randn(1, 64, device="cuda").half()
sf.residual_norm_forward(x, x.clone(), "rms")
r = lambda *s: torch.randn(*s, device="cuda").half() * 0.1
sets = [(r(T, K), r(N, K), r(N)) for T, K, N in ((1, 4096, 1000), (40, 1024, 1024), (250, 8192, 3500), (2500, 1000, 2600))]
def step():
    out = []
    for x, w, b in sets:
        y, s = sf.linear_forward(x, w, b, "gelu", save=True)
        out += [y, *sf.linear_backward(y, s, w)]
    return out + [sf.clip_grad_norm([t.clone() for t in out], 1.0)]
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    held = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(held, step()))
assert sf.dense_error() == 0
"""
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_truth_that_has_none():
    x, w = torch.ones(1, 8, device="cuda").half(), torch.ones(2, 8, device="cuda").half()
    with pytest.raises(RuntimeError):
        sf.linear_forward(x, w, save=torch.ones(2))
