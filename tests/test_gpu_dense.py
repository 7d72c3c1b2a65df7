"""The dense gated FFN, its gradients and the 8-bit activation blocks against plain 64-bit
computations.

Tolerances.  A result is a sum of K products rounded once to its type (half a step:
eps/2 relative), of operands some of which were themselves rounded to the type (H, dG and dU:
eps/2 relative to each term).  Independent roundings of a sum's terms move the sum by at
most eps/2 times the root of its squared terms' sum times a few; a bound that always holds is
eps/2 * sum|terms|.  The fp32 accumulation adds at most (K + 1) 2^-24 sum|terms|.  So
|got - want| <= eps/2 |want| + (stages * eps/2 + K 2^-23) * sum|terms|, with `stages` the
number of rounded intermediates a term passes through, 1 + slack for the next order.
"""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu

KINDS = [torch.float16, torch.bfloat16]


def grid(g, *shape, step=16.0, top=4.0):
    """Normal values on a grid: products of two sum exactly in fp32, so a ReLU's side is certain."""
    return ((torch.randn(*shape, generator=g, device="cuda") * step).round() / step).clamp(-top, top)


def layer(T, d, n, dt, seed=0, bias=True, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    unit = 2.0 ** round(torch.log2(torch.tensor(0.25 / d ** 0.5)).item())
    x = torch.zeros(T, d + pad, device="cuda", dtype=dt)
    x[:, :d] = grid(g, T, d)
    wg = (grid(g, n, d, step=4.0) * 4 * unit).to(dt)
    wu = (torch.randn(n, d, generator=g, device="cuda") / d ** 0.5).to(dt)
    wd = (torch.randn(d, n, generator=g, device="cuda") / n ** 0.5).to(dt)
    b = ((torch.randn(n, generator=g, device="cuda") * 8 - 16).round() / 32).to(dt) if bias else None
    dy = (torch.randn(T, d, generator=g, device="cuda")).to(dt)
    return x[:, :d], wg, wu, wd, b, dy


def near(got, want, terms, dt, stages, K):
    """|got - want| within the bound of the module's docstring (want, terms in 64 bits)."""
    half = torch.finfo(dt).eps / 2
    out = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(dt).smallest_normal  # below it a rounding is absolute
    slack = 1.0 + 4 * half
    tol = slack * (out * want.abs() + (stages * half + K * 2.0 ** -23) * terms) + tiny * (1 + terms.new_tensor(K).sqrt())
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values out of bound, worst " \
                          f"{((got.double() - want).abs() / tol).max().item():.2f} times"


def act8_plain(v, relu):
    T, C = v.shape
    v = torch.nn.functional.pad(v.double(), (0, -C % 64)).view(T, -1, 64)
    if relu:
        v = v.clamp_min(0)
    s = (v.amax(2, keepdim=True) / 255) if relu else v.abs().amax(2, keepdim=True) / 127
    c = (v / s.where(s > 0, torch.ones_like(s))).round()
    if relu:
        c = torch.where((v > 0) & (c < 1), torch.ones_like(c), c)
    return (c * s).view(T, -1)[:, :C], s.expand_as(v).reshape(T, -1)[:, :C]


def forward64(x, wg, wu, wd, b):
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    G = x @ wg.t() + (0 if b is None else b.double())
    U = x @ wu.t()
    return G, U, (G.clamp_min(0) * U)


SHAPES = [(1, 8, 8), (1, 512, 2048), (2, 64, 64), (5, 72, 40), (31, 136, 1000), (128, 64, 256), (129, 200, 264),
          (257, 512, 520), (300, 1000, 1016), (700, 264, 2504)]


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("T,d,n", SHAPES + [(33, 1000, 4096), (40, 520, 1024), (64, 264, 8200), (100, 2048, 4104),
                                            (128, 4096, 2504), (1, 4096, 11008), (3, 1024, 28672), (2, 24, 40000)])
def test_forward(T, d, n, dt):
    x, wg, wu, wd, b, _ = layer(T, d, n, dt, seed=T + d, pad=8 * (T % 3), bias=T % 2 == 1)
    y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b)
    assert saved is None and y.shape == (T, d) and y.dtype == dt
    G, U, H = forward64(x, wg, wu, wd, b)
    terms = (H.abs() + d * 2.0 ** -23 * (x.double().abs() @ wu.double().abs().t()) * G.clamp_min(0)) @ wd.double().abs().t()
    near(y, H @ wd.double().t(), terms, dt, 1, n)
    assert sf.dense_error() == 0


@pytest.mark.parametrize("T,d,n", [(60, 9504, 2048), (100, 9504, 2048), (128, 9504, 2048), (100, 304, 25376),
                                   (48, 8192, 4104), (17, 280, 20312)])
def test_forward_each_product_in_either_kernel(T, d, n):
    """Sizes at which up to 128 tokens take the slim kernel for both products, one or neither."""
    test_forward(T, d, n, torch.float16)


def backward64(x, wg, wu, wd, dy, R, U, on):
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    dH = dy @ wd
    adH = dy.abs() @ wd.abs()
    dU, dG, H = dH * R, dH * U * on, R * U
    adU, adG = adH * R, adH * U.abs() * on
    want = (dG @ wg + dU @ wu, dG.t() @ x, dU.t() @ x, dy.t() @ H, dG.sum(0))
    # terms with each rounded factor's magnitude; the fp32 error of dH rides on adH
    terms = (adG @ wg.abs() + adU @ wu.abs(), adG.t() @ x.abs(), adU.t() @ x.abs(), dy.abs().t() @ H.abs(), adG.sum(0))
    return want, terms


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("T,d,n", SHAPES + [(5000, 1024, 4104), (2100, 1104, 520), (40, 2048, 8)])
def test_backward_full(T, d, n, dt):
    x, wg, wu, wd, b, dy = layer(T, d, n, dt, seed=7 * T + d, bias=T % 2 == 1)
    y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save="full")
    assert torch.equal(y, sf.gated_ffn_forward(x, wg, wu, wd, b)[0])
    G, U, H = forward64(x, wg, wu, wd, b)
    on = (G > 0).double()
    assert torch.equal(saved.r[:, :n] != 0, G > 0), "codes that are not zero are the ReLU's mask"
    got = sf.gated_ffn_backward(dy, saved, wg, wu, wd)
    want, terms = backward64(x, wg, wu, wd, dy, G * on, U, on)
    # a term of dX, dWg, dWu and db passes one rounding (dU or dG), of dWd one (H); the saved
    # codes are off by half a step of the block's largest value, 2^-16 of it, lifted ones by a
    # whole one: counted with the block's largest in place of each value
    def top(v):
        v = torch.nn.functional.pad(v.abs(), (0, -n % 64)).view(T, -1, 64)
        return v.amax(2, keepdim=True).expand_as(v).reshape(T, -1)[:, :n]
    Rt, Ut = top(G * on), top(U)
    adH = dy.double().abs() @ wd.double().abs()
    wg64, wu64, x64 = wg.double().abs(), wu.double().abs(), x.double().abs()
    eG, eU = adH * Ut * on * 2.0 ** -16, adH * Rt * 2.0 ** -16
    extra = (eG @ wg64 + eU @ wu64, eG.t() @ x64, eU.t() @ x64,
             dy.double().abs().t() @ (Rt * U.abs() + Ut * G * on) * 2.0 ** -15, eG.sum(0))
    for i, (g, K) in enumerate(zip(got, (2 * n + d, T + d, T + d, T + d, T + d))):
        if i == 4 and b is None:
            assert g is None
            continue
        near(g, want[i], terms[i] + extra[i] / (torch.finfo(dt).eps / 2), dt, 1, K)
    assert sf.dense_error() == 0


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("T,d,n", SHAPES)
def test_backward_act8(T, d, n, dt):
    x, wg, wu, wd, b, dy = layer(T, d, n, dt, seed=3 * T + d, bias=T % 2 == 1)
    y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save="act8")
    assert torch.equal(y, sf.gated_ffn_forward(x, wg, wu, wd, b)[0])
    G, U, _ = forward64(x, wg, wu, wd, b)
    on = (G > 0).double()
    assert torch.equal((saved.r > 0)[:, :n], G > 0), "codes above zero are the ReLU's mask"
    # the held values against the formula: half a code, and a whole one where a small positive
    # value was lifted to code 1 (U is an fp32 sum: K 2^-23 of its terms more)
    R8 = saved.r[:, :n].double() * saved.r_scales.double().repeat_interleave(64, 1)[:, :n]
    U8 = saved.u.view(torch.int8)[:, :n].double() * saved.u_scales.double().repeat_interleave(64, 1)[:, :n]
    X8 = saved.x_codes.view(torch.int8)[:, :d].double() * saved.x_scales.double().repeat_interleave(64, 1)[:, :d]
    for held, v, relu in ((R8, G, True), (U8, U, False), (X8, x.double(), False)):
        want, s = act8_plain(v, relu)
        slack = d * 2.0 ** -23 * (x.double().abs() @ (wu.double().abs()).t()) if v is U else 0
        lifted = (held > 0) & (v < 0.5 * s) if relu else torch.zeros_like(s, dtype=torch.bool)
        err = (held - (v.clamp_min(0) if relu else v)).abs()
        assert (err <= torch.where(lifted, s, 0.5 * s) * (1 + 2.0 ** -10) + slack + 1e-30).all()
    got = sf.gated_ffn_backward(dy, saved, wg, wu, wd)
    want, terms = backward64(X8, wg, wu, wd, dy, R8, U8, on)  # the gradients' formula on the held values
    for i, (g, K) in enumerate(zip(got, (2 * n + d, T + d, T + d, T + d, T + d))):
        if i == 4 and b is None:
            continue
        near(g, want[i], terms[i], dt, 2, K)  # X restored (or H) and dU or dG rounded
    assert sf.dense_error() == 0


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("relu", [False, True])
@pytest.mark.parametrize("T,C", [(1, 1), (1, 64), (3, 65), (2, 127), (7, 1000), (33, 2048), (9, 2049), (4, 11008), (1, 28672)])
def test_act8_blocks(T, C, relu, dt):
    g = torch.Generator(device="cuda").manual_seed(T * 31 + C)
    x = (torch.randn(T, C, generator=g, device="cuda") * 3).to(dt)
    x[0, : C // 2] = 0  # whole zero blocks
    q = sf.quantize_act8(x, relu=relu)
    got = sf.dequantize_act8(q)
    want, s = act8_plain(x, relu)
    v = x.double().clamp_min(0) if relu else x.double()
    lifted = (v > 0) & (v < 0.5 * s) if relu else torch.zeros_like(s, dtype=torch.bool)
    bound = torch.where(lifted, s, 0.5 * s) * (1 + 2.0 ** -10) + want.abs() * torch.finfo(dt).eps / 2 * 1.01
    assert ((got.double() - v).abs() <= bound + torch.finfo(dt).smallest_normal).all()
    if relu:
        assert torch.equal((q.codes > 0)[:, :C], x > 0)
    assert (q.codes[:, C:] == 0).all()
    # rows of a wider tensor, unaligned base
    wide = torch.zeros(T, C + 3, dtype=dt, device="cuda")
    wide[:, 1: C + 1] = x
    q2 = sf.quantize_act8(wide[:, 1: C + 1], relu=relu)
    assert torch.equal(q2.codes, q.codes) and torch.equal(q2.scales, q.scales)
    out = torch.full((T, C + 3), 7.0, dtype=dt, device="cuda")
    sf.dequantize_act8(q, out=out[:, 1: C + 1])
    assert torch.equal(out[:, 1: C + 1], got) and (out[:, 0] == 7).all() and (out[:, C + 1:] == 7).all()


@pytest.mark.parametrize("relu", [False, True])
def test_act8_special_values(relu):
    x = torch.ones(6, 130, device="cuda", dtype=torch.bfloat16)
    x[0, 3] = float("nan")
    x[1, 70] = float("inf")
    x[2, 129] = float("-inf")
    x[3] = 2.0 ** -122  # below the smallest scale
    x[4] = 3e38
    x[5, 5] = 1e-30  # positive beside ones
    y = sf.dequantize_act8(sf.quantize_act8(x, relu=relu)).float()
    assert y[0, :64].isnan().all() and (y[0, 64:] == 1).all()
    assert y[1, 64:128].isnan().all() and (y[1, :64] == 1).all()
    if relu:
        assert (y[2, 128] == 1) and y[2, 129] == 0
    else:
        assert y[2, 128:].isnan().all()
    assert (y[3] == 0).all()
    assert ((y[4] - x[4].float()).abs() <= 2.0 ** -8 * x[4].float()).all()
    assert y[5, 5] == (torch.tensor(1 / 255.0).bfloat16().item() if relu else 0)


def test_autograd_matches_the_explicit_calls_and_differences():
    dt = torch.float16
    x, wg, wu, wd, b, dy = layer(40, 64, 128, dt, seed=1)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu, wd, b)]
    for checkpoint in ("full", "act8"):
        y = sf.gated_ffn(leaves[0].view(5, 8, 64), *leaves[1:], checkpoint=checkpoint)
        assert y.shape == (5, 8, 64)
        grads = torch.autograd.grad(y, leaves, dy.view(5, 8, 64))
        y2, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save=checkpoint)
        want = sf.gated_ffn_backward(dy, saved, wg, wu, wd)
        assert torch.equal(y.reshape(40, 64), y2)
        for a, c in zip(grads, want):
            assert torch.equal(a, c)
    # differences of the 64-bit formula along a direction, against the "full" gradients
    y = sf.gated_ffn(*leaves)
    grads = torch.autograd.grad(y, leaves, dy)
    g = torch.Generator(device="cuda").manual_seed(5)
    for i, leaf in enumerate(leaves):
        v = torch.randn(leaf.shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-7  # no gate sum lies within its reach of the ReLU's border: they sit on a grid
        def loss(sgn):
            p = [t.detach().double() for t in leaves]
            p[i] = p[i] + sgn * h * v
            G, U = p[0] @ p[1].t() + p[4], p[0] @ p[2].t()
            off = (leaves[0].detach().double() @ leaves[1].detach().double().t() + leaves[4].detach().double()) <= 0
            return ((G.masked_fill(off, 0) * U) @ p[3].t() * dy.double()).sum()
        slope = (loss(1) - loss(-1)) / (2 * h)
        dot = (grads[i].double() * v).sum()
        # each gradient element is off by a few roundings of its own size or of its terms' size:
        # random in sign, so their sum along v moves by at most 8 eps times the 2-norm
        scale = (grads[i].double() * v).norm() + grads[i].double().norm()
        assert abs(slope - dot) <= 8 * torch.finfo(dt).eps * scale + 1e-5 * scale


def test_shapes_views_and_no_grad():
    x, wg, wu, wd, b, dy = layer(24, 64, 128, torch.bfloat16, seed=2)
    want = sf.gated_ffn_forward(x, wg, wu, wd, b)[0]
    with torch.no_grad():
        assert torch.equal(sf.gated_ffn(x.view(2, 3, 4, 64), wg, wu, wd, b).view(24, 64), want)
    assert torch.equal(sf.gated_ffn_forward(x[0], wg, wu, wd, b)[0], sf.gated_ffn_forward(x[:1], wg, wu, wd, b)[0][0])
    wide = torch.randn(128, 64 + 16, device="cuda").to(torch.bfloat16)
    wide[:, 8:72] = wg
    assert torch.equal(sf.gated_ffn_forward(x, wide[:, 8:72], wu, wd, b)[0], want)
    for shape in ((0, 64), (3, 0, 64)):
        e = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        for save in ("full", "act8"):
            y, saved = sf.gated_ffn_forward(e, wg, wu, wd, b, save=save)
            assert y.shape == shape
            g = sf.gated_ffn_backward(torch.empty_like(e), saved, wg, wu, wd)
            assert g[0].shape == shape and all((t == 0).all() for t in g[1:])
    # gradients that are not needed are not computed
    y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save="full")
    all_of = sf.gated_ffn_backward(dy, saved, wg, wu, wd)
    for i in range(5):
        need = [j == i for j in range(5)]
        some = sf.gated_ffn_backward(dy, saved, wg, wu, wd, need=need)
        assert all((some[j] is None) == (j != i) for j in range(5)) and torch.equal(some[i], all_of[i])
    # an expanded gradient (a sum's) arrives with zero strides
    leaf = wg.clone().requires_grad_()
    g1 = torch.autograd.grad(sf.gated_ffn(x, leaf, wu, wd, b).sum(), leaf)[0]
    g2 = sf.gated_ffn_backward(torch.ones_like(dy), saved, wg, wu, wd)[1]
    assert torch.equal(g1, g2)


def test_nan_and_infinity_stay_in_their_token():
    x, wg, wu, wd, b, dy = layer(300, 64, 128, torch.bfloat16, seed=3)
    want = sf.gated_ffn_forward(x, wg, wu, wd, b)[0]
    x2 = x.clone()
    x2[7, 3] = float("nan")
    x2[260, 1] = float("inf")
    got = sf.gated_ffn_forward(x2, wg, wu, wd, b)[0]
    assert got[7].isnan().all() and not got[260].isfinite().any()
    rest = [t for t in range(300) if t not in (7, 260)]
    assert torch.equal(got[rest], want[rest])


def test_streams_graphs_and_repeats():
    x, wg, wu, wd, b, dy = layer(200, 256, 512, torch.bfloat16, seed=4)

    def step(save):
        y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save=save)
        return (y,) + sf.gated_ffn_backward(dy, saved, wg, wu, wd)

    want = {k: [t.clone() for t in step(k)] for k in ("full", "act8")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = sf.gated_ffn_forward(x, wg, wu, wd, b, stream=side)[0]
    side.synchronize()
    assert torch.equal(y, want["full"][0])
    # two captured steps replayed in turn, several times, with other inputs in between
    graphs = {}
    for k in ("full", "act8"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(k)
        graphs[k] = (g, out)
    keep = x.clone()
    for k in ("full", "act8", "act8", "full"):
        x.mul_(0.5)
        graphs[k][0].replay()
        x.copy_(keep)
        graphs[k][0].replay()
        torch.cuda.synchronize()
        for a, c in zip(graphs[k][1], want[k]):
            assert torch.equal(a, c)
    # steps on two streams at once
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for s, k in zip(streams, ("full", "act8")):
            with torch.cuda.stream(s):
                outs.append((k, step(k)))
    torch.cuda.synchronize()
    for k, out in outs:
        for a, c in zip(out, want[k]):
            assert torch.equal(a, c)
    assert sf.dense_error() == 0


@pytest.mark.parametrize("act", ["reglu", "relu"])
@pytest.mark.parametrize("d,n", [(512, 1000), (256, 2051), (128, 72)])
def test_prompt_through_a_handle(act, d, n):
    import workload as W
    cfg = W.small_config(W.CONFIGS["70b_reglu" if act == "reglu" else "opt6.7b_relu"], d=d, n=n, r=64)
    lay = W.make_layer(cfg, seed=3)
    h = sf.SparseFFN.from_layer(lay, max_batch=2, device="cuda:0")
    to64 = lambda a: torch.from_numpy(a).cuda().double()
    for T in (1, 2, 33, 300):
        X = torch.randn(T, d, generator=torch.Generator().manual_seed(T)).half().cuda()
        Y = h.forward_prompt(X)
        x, wu, wd, b = X.double(), to64(lay.w_up), to64(lay.w_down), to64(lay.b)
        U = x @ wu.t()
        first = x @ to64(lay.w_gate).t() + b if act == "reglu" else U + b
        H = first.clamp_min(0) * (U if act == "reglu" else 1)
        # fp32 sums of both products, H rounded to fp16 (near the ReLU's border a wrong side
        # costs no more than the fp32 error of the sum)
        slack = d * 2.0 ** -23 * ((x.abs() @ wu.abs().t()) * (first.clamp_min(0) if act == "reglu" else 1))
        if act == "reglu":
            slack = slack + d * 2.0 ** -23 * (x.abs() @ to64(lay.w_gate).abs().t()) * U.abs()
        half = torch.finfo(torch.float16).eps / 2
        tol = ((half * 1.01 + n * 2.0 ** -23) * H.abs() + slack + 2.0 ** -25) @ wd.abs().t() + 2.0 ** -23 * (H @ wd.t()).abs()
        assert ((Y.double() - H @ wd.t()).abs() <= tol).all()
        # every neuron: the sparse step over an explicit full set agrees (single token)
        if T == 1:
            y = h.forward(X[0], idx=torch.arange(n, dtype=torch.int32, device="cuda"))
            assert ((y.double() - Y[0].double()).abs() <= 2 * tol[0] + 2e-3 * Y.abs().max()).all()
    assert h.forward_prompt(torch.empty(0, d, device="cuda", dtype=torch.float16)).shape == (0, d)
    assert h.get_error() == 0
    h.close()
    if d % 32 == 0:
        hq = sf.SparseFFN.from_layer(lay, device="cuda:0", rows="int8")
        with pytest.raises(sf.SfnnError) as e:
            hq.forward_prompt(X)
        assert e.value.status == sf.STATUS_CODES["SFNN_ERR_UNSUPPORTED"]
        hq.close()


def test_autograd_captured_in_a_graph():
    """Forward and torch.autograd.grad captured together, as a training loop would."""
    x, wg, wu, wd, b, dy = layer(48, 64, 128, torch.bfloat16, seed=9)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu, wd, b)]
    want = [t.clone() for t in torch.autograd.grad(sf.gated_ffn(*leaves, checkpoint="act8"), leaves, dy)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(sf.gated_ffn(*leaves, checkpoint="act8"), leaves, dy)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grads = torch.autograd.grad(sf.gated_ffn(*leaves, checkpoint="act8"), leaves, dy)
    for _ in range(2):
        for t in grads:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, c in zip(grads, want):
            assert torch.equal(a, c)
    assert sf.dense_error() == 0


def test_offsets_beyond_32_bits():
    """Hidden layers of more than 2^31 elements; checked at tokens and neurons at both ends."""
    T, d, n, dt = 70001, 64, 32768, torch.bfloat16
    assert T * n > 2 ** 31
    x, wg, wu, wd, b, dy = layer(T, d, n, dt, seed=10)
    y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save="full")
    rows = torch.tensor([0, 1, 35000, T - 257, T - 2, T - 1], device="cuda")
    G, U, H = forward64(x[rows], wg, wu, wd, b)
    near(y[rows], H @ wd.double().t(), H.abs() @ wd.double().abs().t(), dt, 1, n)
    dx, dwg, dwu, dwd, db = sf.gated_ffn_backward(dy, saved, wg, wu, wd)
    del saved
    on = (G > 0).double()
    (wdx, *_), (tdx, *_) = backward64(x[rows], wg, wu, wd, dy[rows], G * on, U, on)
    near(dx[rows], wdx, 1.02 * tdx, dt, 1, 2 * n + d)
    cols = torch.tensor([0, 77, n // 2, n - 65, n - 1], device="cuda")
    Gc, Uc, Hc = forward64(x, wg[cols], wu[cols], wd[:, cols], b[cols])
    onc = (Gc > 0).double()
    want, terms = backward64(x, wg[cols], wu[cols], wd[:, cols], dy, Gc * onc, Uc, onc)
    near(dwg[cols], want[1], 1.02 * terms[1], dt, 1, T + d)
    near(dwu[cols], want[2], 1.02 * terms[2], dt, 1, T + d)
    near(dwd[:, cols], want[3], 1.02 * terms[3], dt, 1, T + d)
    near(db[cols], want[4], 1.02 * terms[4], dt, 1, T + d)
    del dx, dwg, dwu, dwd, db, y
    C = 32768
    big = torch.zeros(T, C, dtype=dt, device="cuda")
    big[rows] = torch.randn(6, C, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dt)
    q = sf.quantize_act8(big)
    few = sf.dequantize_act8(sf.quantize_act8(big[rows].contiguous()))
    out = sf.dequantize_act8(q)
    assert torch.equal(out[rows], few) and int((out != 0).any(1).sum()) == 6
    assert sf.dense_error() == 0


def test_refusals():
    x, wg, wu, wd, b, dy = layer(16, 64, 128, torch.float16, seed=11)
    ok = lambda **k: sf.gated_ffn_forward(*[k.get(n, t) for n, t in
                                            (("x", x), ("wg", wg), ("wu", wu), ("wd", wd), ("b", b))])
    ok()
    for err, k in ((TypeError, dict(x=x.float())), (TypeError, dict(wg=wg.bfloat16())), (TypeError, dict(wd=wd.cpu())),
                   (ValueError, dict(x=x[:, :56])), (ValueError, dict(wu=wu[:64])), (ValueError, dict(wd=wd.t())),
                   (ValueError, dict(b=b[:64])), (ValueError, dict(b=b.float())), (ValueError, dict(x=x.t())),
                   (ValueError, dict(x=x[:1].expand(16, 64))),
                   (ValueError, dict(x=torch.zeros(16 * 64 + 4, dtype=x.dtype, device="cuda")[4:].view(16, 64))),
                   (ValueError, dict(wg=torch.zeros(128, 68, dtype=x.dtype, device="cuda")[:, 4:]))):
        with pytest.raises(err):
            ok(**k)
    with pytest.raises(ValueError):  # widths in steps of 8
        sf.gated_ffn_forward(x[:, :60].contiguous(), wg[:, :60].contiguous(), wu[:, :60].contiguous(), wd[:60].contiguous())
    _, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save="full")
    with pytest.raises(ValueError):
        sf.gated_ffn_backward(dy[:8], saved, wg, wu, wd)
    with pytest.raises(TypeError):
        sf.gated_ffn_backward(dy.float(), saved, wg, wu, wd)
    w = x.clone().requires_grad_()
    y = sf.gated_ffn(w * 1, wg, wu, wd, b)
    with torch.no_grad():
        q = sf.quantize_mxfp4(wg)
    with pytest.raises(ValueError):
        sf.mxfp4_linear(x[:, :32], q)
    with pytest.raises(ValueError):
        sf.quantize_mxfp4(x[:, :48].contiguous())
    with pytest.raises(TypeError):
        sf.mxfp4_linear(x, q, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        sf.dequantize_act8(sf.quantize_act8(x), out=torch.empty(16, 63, dtype=x.dtype, device="cuda"))
    y.sum().backward()
    assert w.grad is not None and sf.dense_error() == 0


def test_a_weight_changed_between_the_passes_is_noticed():
    x, wg, wu, wd, b, dy = layer(16, 64, 128, torch.float16, seed=12)
    wg = wg.requires_grad_()
    y = sf.gated_ffn(x, wg, wu, wd, b)
    with torch.no_grad():
        wg.mul_(2.0)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, wg, dy)
