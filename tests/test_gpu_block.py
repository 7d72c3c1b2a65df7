"""The norms around a block and the clipping of gradients against plain 64-bit computations.

Tolerances.  A result is computed in 32 bits and rounded once to its type: half a step (eps / 2 of
the value), plus the 32-bit errors.  Those are at most a few 2^-24 of each term that enters the
result, where a row's mean and deviation are sums of d values: a thread adds up at most 16 of them
one after the other, and the rest is a tree of at most 12 more levels and 128 parts' sums, so 2^-24
times 156 covers a sum and 2^-24 times 400 a value that passes through two of them and a handful of
products.  ``terms`` is each result with every term's magnitude in the place of the term.  A sum
over T rows adds T 2^-24 of its terms."""
import math

import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu

KINDS = [torch.float16, torch.bfloat16]
EPS = 1e-5
FP32 = 400 * 2.0 ** -24


def near(got, want, terms, K=0):
    """|got - want| within half a step of got's type and the 32-bit errors of the module's docstring."""
    info = torch.finfo(got.dtype)
    tol = info.eps / 2 * want.abs() + (FP32 + K * 2.0 ** -24) * terms + info.smallest_normal * info.eps
    bad = ~((got.double() - want).abs() <= tol * 1.001)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} out of bound, worst " \
                          f"{((got.double() - want).abs() / tol).max().item():.2f} times"


def inputs(T, d, dt, seed=0, z=True, gate=None, pre="rms", post="none", bias=False, x32=False, z32=False, pad=0, off=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")

    def rows(v, dtype):  # T rows in a wider buffer that starts `off` values in
        buf = torch.full((T * (d + pad) + off,), 7.0, device="cuda", dtype=dtype)
        view = buf[off:].view(T, d + pad)[:, :d]
        view.copy_(v)
        return view
    a = {"x": rows(r(T, d) * 2 + 0.3, torch.float32 if x32 else dt),
         "z": rows(r(T, d) * torch.exp(r(T, 1)), torch.float32 if z32 else dt) if z else None,
         "gate": {None: None, "vec": (1 + 0.3 * r(d)).to(dt), "token": rows(r(T, d), dt)}[gate]}
    for k, kind in (("", pre), ("post_", post)):
        a[k + "w"] = (1 + 0.2 * r(d)).to(dt) if kind != "none" else None
        a[k + "b"] = (0.2 * r(d)).to(dt) if kind != "none" and bias else None
    return a, (lambda dtype: rows(r(T, d) * 0.3, dtype))


def normed(v, at, kind):
    """(v^, 1/deviation, magnitude of v^'s terms) from v and its terms' magnitudes."""
    m = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    ma = at.mean(1, keepdim=True) if kind == "layer" else m
    s = 1 / ((v - m).square().mean(1, keepdim=True) + EPS).sqrt()
    # the deviation's own error: of the squares' terms, relative to their sum
    rel = ((at + ma).square().mean(1, keepdim=True) * s * s).clamp_min(1.0)
    return (v - m) * s, s, (at + ma) * s * rel


def plain(a, pre, post, A=1.0, C=1.0, dr=None, dh=None):
    """R, H and the gradients in 64 bits, with their terms' magnitudes, from the formulas."""
    f = {k: None if v is None else v.double() for k, v in a.items()}
    one = lambda v, o: o if v is None else v
    x, z, g = f["x"], f["z"], one(f["gate"], 1.0)
    ga = abs(g) if isinstance(g, float) else g.abs()
    if z is None:
        r, ra = x, x.abs()
    else:
        zh, zs, zha = (z, 1.0, z.abs()) if post == "none" else normed(z, z.abs(), post)
        wp, bp = one(f["post_w"], 1.0), one(f["post_b"], 0.0)
        wpa = abs(wp) if isinstance(wp, float) else wp.abs()
        p, pa = zh * wp + bp, zha * wpa + (abs(bp) if isinstance(bp, float) else bp.abs())
        r, ra = A * x + C * g * p, abs(A) * x.abs() + abs(C) * ga * pa
    out = {"r": (r, ra)}
    if pre != "none":
        rh, rs, rha = normed(r, ra, pre)
        w, b = one(f["w"], 1.0), one(f["b"], 0.0)
        wa = abs(w) if isinstance(w, float) else w.abs()
        out["h"] = (rh * w + b, rha * wa + (abs(b) if isinstance(b, float) else b.abs()))
    if dr is None and dh is None:
        return out
    zero = torch.zeros_like(x)
    D = zero if dr is None else dr.double()
    Da = D.abs()

    def back(u, ua, hat, hata, s, kind):
        v = u - hat * (u * hat).mean(1, keepdim=True)
        # s and hat carry hata's relative errors; each appears with its own magnitude
        va = ua + hata * (ua * hata).mean(1, keepdim=True)
        grow = (hata.square().mean(1, keepdim=True)).clamp_min(1.0)
        if kind == "layer":
            v, va = v - u.mean(1, keepdim=True), va + ua.mean(1, keepdim=True)
        return s * v, s * va * grow
    if dh is not None:
        dh = dh.double()
        out["w"], out["b"] = ((dh * rh).sum(0), (dh.abs() * rha).sum(0)), (dh.sum(0), dh.abs().sum(0))
        v, va = back(dh * w, dh.abs() * wa, rh, rha, rs, pre)
        D, Da = D + v, Da + va
    out["x"] = (A * D, abs(A) * Da) if z is not None else (D, Da)
    if z is not None:
        q, qa = C * D, abs(C) * Da
        out["gate"] = (q * p, qa * pa)
        if f["gate"] is not None and f["gate"].dim() == 1:
            out["gate"] = tuple(t.sum(0) for t in out["gate"])
        q, qa = q * g, qa * ga
        if post != "none":
            out["post_w"], out["post_b"] = ((q * zh).sum(0), (qa * zha).sum(0)), (q.sum(0), qa.sum(0))
            q, qa = back(q * wp, qa * wpa, zh, zha, zs, post)
        out["z"] = (q, qa)
    return out


def call(a, pre, post, save=False, **kw):
    return sf.residual_norm_forward(a["x"], a["z"], pre, a["w"], a["b"], post, a["post_w"], a["post_b"], a["gate"],
                                    eps=EPS, save=save, **kw)


GRADS = ["x", "z", "gate", "w", "b", "post_w", "post_b"]


def check(T, d, dt, A=1.0, C=1.0, seed=0, **kw):
    a, rows = inputs(T, d, dt, seed=seed, **kw)
    pre, post = kw.get("pre", "rms"), kw.get("post", "none")
    r, h, saved = call(a, pre, post, save=True, residual_scale=A, branch_scale=C, dtype=dt)
    assert r.dtype == a["x"].dtype and (h is None) == (pre == "none") and (h is None or h.dtype == dt)
    dr, dh = rows(a["x"].dtype), rows(dt) if pre != "none" else None
    want = plain(a, pre, post, A, C, dr, dh)
    near(r, *want["r"]) if a["z"] is not None else None
    assert r is a["x"] or a["z"] is not None
    if h is not None:
        near(h, *want["h"])
    # without saving: the same to the bit
    again = call(a, pre, post, residual_scale=A, branch_scale=C, dtype=dt)
    assert again[2] is None and torch.equal(again[0], r) and (h is None or torch.equal(again[1], h))
    got = dict(zip(GRADS, sf.residual_norm_backward(dr, dh, saved)))
    for k, v in got.items():
        assert (v is None) == (a[k] is None), k
        if v is not None:
            assert v.dtype == a[k].dtype and v.shape == a[k].shape
            near(v, *want[k], K=T if v.dim() == 1 else 0)
    once = sf.residual_norm_backward(dr, dh, saved)
    assert all(u is None or torch.equal(u, v) for u, v in zip(once, got.values()))
    return a, rows, saved


WIDTHS = [1, 2, 7, 8, 31, 33, 256, 257, 264, 1000, 1001, 1024, 2047, 4096, 4097, 4104, 5000, 8192]


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(d, dt):
    kinds = ["none", "rms", "layer"]
    check(5, d, dt, seed=d, pre=kinds[1 + d % 2], post=kinds[d % 3], gate=[None, "vec", "token"][d % 3],
          bias=d % 2 == 0, x32=d % 5 < 2, z32=d % 7 < 2)


@pytest.mark.parametrize("d", [8193, 8200, 12000, 16384, 16385, 32767, 32768])
def test_wide_rows_over_several_ctas(d):
    check(3, d, KINDS[d % 2], seed=d, pre="layer", post="rms", gate="vec", bias=True)
    check(2, d, KINDS[d % 2], seed=d, pre="rms", z=False)


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate", [None, "vec", "token"])
def test_kinds(gate, post, pre, dt):
    for i, (T, d) in enumerate(((37, 264), (6, 129))):
        check(T, d, dt, A=0.75, C=-0.5, seed=T, pre=pre, post=post, gate=gate, bias=i == 0, x32=i == 1, z32=gate == "vec")


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("T", [1, 2, 3, 4, 9, 300, 2500])
def test_token_counts(T, dt):
    check(T, 512, dt, seed=T, pre="rms", post="rms", gate="vec")
    check(T, 100, dt, seed=T, pre="layer", z=False, bias=True, x32=True)


@pytest.mark.parametrize("pad,off", [(8, 0), (64, 8), (1, 0), (3, 1), (0, 1), (4, 4)])
def test_strides_and_alignments(pad, off):
    for x32 in (False, True):
        check(11, 1000, torch.bfloat16, pre="rms", post="layer", gate="token", bias=True, pad=pad, off=off, x32=x32)


def test_leading_dimensions_and_no_tokens():
    a, _ = inputs(12, 64, torch.float16, post="rms", gate="vec")
    r, h, _ = call(a, "rms", "rms")
    b = {k: v.view(3, 4, 64) if k in ("x", "z") else v for k, v in a.items()}
    r3, h3, saved = call(b, "rms", "rms", save=True)
    assert torch.equal(r3.view(12, 64), r) and torch.equal(h3.view(12, 64), h) and r3.shape == (3, 4, 64)
    v = {k: v[0] if k in ("x", "z") else v for k, v in a.items()}
    r1, h1, _ = call(v, "rms", "rms")
    assert torch.equal(r1, r[0]) and torch.equal(h1, h[0])
    e = {k: v[:0] if k in ("x", "z") else v for k, v in a.items()}
    r0, h0, saved = call(e, "rms", "rms", save=True)
    assert r0.shape == h0.shape == (0, 64)
    g = sf.residual_norm_backward(r0, h0, saved)
    assert g[0].shape == (0, 64) and all((t == 0).all() for t in (g[2], g[3], g[5]))


@pytest.mark.parametrize("dt", KINDS)
def test_rows_of_zeros_large_values_and_values_that_are_not_finite(dt):
    a, rows = inputs(6, 136, dt, pre="layer", post="rms", bias=True)
    a["x"][0], a["z"][0] = 0, 0          # a row of nothing: the norms divide by sqrt(eps)
    a["z"][1, 3] = float("nan")
    a["x"][2, 5] = float("inf")
    a["x"][3], a["z"][3] = torch.finfo(dt).max / 2, 1.0  # equal large values
    r, h, saved = call(a, "layer", "rms", save=True)
    want = plain(a, "layer", "rms")
    for i in (0, 4, 5):
        near(r[i], want["r"][0][i], want["r"][1][i]), near(h[i], want["h"][0][i], want["h"][1][i])
    assert h[1].isnan().all() and r[1].isnan().all()  # the post norm's row; then all of the pre norm's
    assert r[2, 5].isinf() and h[2].isnan().all()
    if dt == torch.float16:
        assert torch.isfinite(h[3]).all()
    dr, dh = rows(dt), rows(dt)
    got = sf.residual_norm_backward(dr, dh, saved)
    assert torch.isfinite(got[0][[0, 4, 5]]).all() and torch.isfinite(got[1][[0, 4, 5]]).all()
    assert got[0][1].isnan().all() and got[3].isnan().all()


def test_gradients_that_are_left_out_and_missing_ones():
    a, rows = inputs(40, 264, torch.bfloat16, pre="rms", post="layer", gate="vec", bias=True)
    r, h, saved = call(a, "rms", "layer", save=True)
    dr, dh = rows(torch.bfloat16), rows(torch.bfloat16)
    zero = torch.zeros_like(dr)
    full = sf.residual_norm_backward(dr, dh, saved)
    for i in range(7):
        need = [j == i for j in range(7)]
        got = sf.residual_norm_backward(dr, dh, saved, need=need)
        assert all((t is None) == (j != i) for j, t in enumerate(got)) and torch.equal(got[i], full[i])
    for u, v in zip(sf.residual_norm_backward(None, dh, saved), sf.residual_norm_backward(zero, dh, saved)):
        assert torch.equal(u, v)
    for u, v in zip(sf.residual_norm_backward(dr, None, saved), sf.residual_norm_backward(dr, zero, saved)):
        assert torch.equal(u, v)


@pytest.mark.parametrize("pre,post,gate", [("rms", "rms", "vec"), ("layer", "layer", "token"), ("rms", "none", None)])
def test_gradients_against_differences(pre, post, gate):
    """Along random directions, against central differences of the 64-bit formulas."""
    a, rows = inputs(5, 40, torch.bfloat16, pre=pre, post=post, gate=gate, bias=True, x32=True, z32=True)
    dr, dh = rows(torch.float32), rows(torch.bfloat16)
    r, h, saved = call(a, pre, post, save=True, dtype=torch.bfloat16)
    got = dict(zip(GRADS, sf.residual_norm_backward(dr, dh, saved)))
    want = plain(a, pre, post, dr=dr, dh=dh)
    g = torch.Generator(device="cuda").manual_seed(3)

    def loss(v):
        o = plain(v, pre, post)
        return (o["r"][0] * dr.double()).sum() + (o["h"][0] * dh.double()).sum()
    for k in GRADS:
        if a[k] is None:
            continue
        v = torch.randn(a[k].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-5
        up, down = ({**{n: None if t is None else t.double() for n, t in a.items()}, k: a[k].double() + s * v}
                    for s in (step, -step))
        slope = (loss(up) - loss(down)) / (2 * step)
        # got is off by half a step of its type, the differences by step^2 of the third derivative
        tol = (torch.finfo(got[k].dtype).eps / 2 * got[k].double().abs() + FP32 * want[k][1]) * v.abs()
        assert abs((got[k].double() * v).sum() - slope) <= tol.sum() + 1e-6 * (1 + abs(slope)), k


def test_autograd():
    a, rows = inputs(9, 72, torch.float16, pre="rms", post="rms", gate="vec")
    leaves = {k: v.clone().requires_grad_() for k, v in a.items() if v is not None}
    r, h = sf.residual_norm(leaves["x"], leaves["z"], "rms", leaves["w"], post="rms", post_w=leaves["post_w"],
                            gate=leaves["gate"], eps=EPS)
    r0, h0, saved = call(a, "rms", "rms", save=True)
    assert torch.equal(r, r0) and torch.equal(h, h0)
    dr, dh = rows(torch.float16), rows(torch.float16)
    got = torch.autograd.grad([r, h], list(leaves.values()), [dr, dh], retain_graph=True)
    want = dict(zip(GRADS, sf.residual_norm_backward(dr, dh, saved)))
    for k, v in zip(leaves, got):
        assert torch.equal(v, want[k])
    # one of the two outputs alone, with an expanded gradient
    (gx,) = torch.autograd.grad(h.float().sum(), leaves["x"], retain_graph=True)
    assert torch.equal(gx, sf.residual_norm_backward(None, torch.ones_like(h), saved)[0])
    (gx,) = torch.autograd.grad(r.sum(), leaves["x"])
    assert torch.equal(gx, torch.ones_like(gx))
    # without z the residual is x itself, and its gradient adds up
    x = a["x"].clone().requires_grad_()
    r, h = sf.residual_norm(x, w=a["w"])
    assert r is x
    (gx,) = torch.autograd.grad((r.float() * 2).sum() + h.float().sum(), x)
    _, _, saved = sf.residual_norm_forward(a["x"], w=a["w"], save=True)
    alone = sf.residual_norm_backward(None, torch.ones_like(h), saved)[0]
    assert torch.equal(gx, alone + 2)
    # only a post norm
    x, z = a["x"].clone().requires_grad_(), a["z"].clone().requires_grad_()
    r, h = sf.residual_norm(x, z, "none", post="rms")
    assert h is None
    gx, gz = torch.autograd.grad(r, (x, z), dr)
    assert torch.equal(gx, dr) and gz.shape == z.shape
    with pytest.raises(RuntimeError):  # twice is refused
        gx, = torch.autograd.grad(sf.residual_norm(x, z)[1].sum(), x, create_graph=True)
        gx.sum().backward()
    with torch.no_grad():
        assert not sf.residual_norm(x, z)[0].requires_grad


def test_in_place_residual_and_other_streams():
    a, _ = inputs(50, 520, torch.bfloat16, pre="rms", x32=True, z32=True)
    r, h, _ = call(a, "rms", "none")
    x = a["x"].clone()
    r2, h2, _ = call({**a, "x": x}, "rms", "none", out=x)
    assert r2 is x and torch.equal(x, r) and torch.equal(h2, h)
    with pytest.raises(ValueError):
        call({**a, "x": x}, "rms", "none", out=x, save=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r3, h3, saved = call(a, "rms", "none", save=True, stream=side)
    got = sf.residual_norm_backward(r, h, saved, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r3, r) and torch.equal(h3, h)
    _, _, saved = call(a, "rms", "none", save=True)
    for u, v in zip(got, sf.residual_norm_backward(r, h, saved)):
        assert u is v is None or torch.equal(u, v)


def test_norms_in_a_graph():
    a, rows = inputs(33, 264, torch.float16, pre="rms", post="rms", gate="vec")
    dr, dh = rows(torch.float16), rows(torch.float16)

    def step():
        r, h, saved = call(a, "rms", "rms", save=True)
        return [r, h] + [t for t in sf.residual_norm_backward(dr, dh, saved) if t is not None]
    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        a["x"].copy_(torch.randn(33, 264, generator=gen, device="cuda"))
        dh.copy_(torch.randn(33, 264, generator=gen, device="cuda"))
        for g in graphs:
            g.replay()
        for out in outs:
            for u, v in zip(out, step()):
                assert torch.equal(u, v)


# ------------------------------------------------------------------ clipping
def grads_of(sizes, dtypes, seed=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=g, device="cuda") * size).to(dt) for s, dt in zip(sizes, dtypes)]


def clip64(grads, max_norm, scale=1.0, eps=1e-6):
    n = scale * math.sqrt(sum(g.double().square().sum().item() for g in grads))
    return n, scale * min(1.0, max_norm / (n + eps))


def check_clip(grads, max_norm, scale=1.0, out=None):
    before = [g.clone() for g in grads]
    n, k = clip64(grads, max_norm, scale)
    norm = sf.clip_grad_norm(grads, max_norm, scale=scale, out=out)
    assert norm.dtype == torch.float32 and norm.shape == ()
    # sums of up to 8 squares in 32 bits, then 64; the root halves their error; one rounding
    assert abs(norm.item() - n) <= 2.0 ** -20 * n
    for b, o, g in zip(before, out or grads, grads):
        want = b.double() * k
        info = torch.finfo(b.dtype)
        # k: n's error, a sum, a quotient and a product in 32 bits; then one product and the type's rounding
        tol = (info.eps / 2 + 2.0 ** -19) * want.abs() + info.smallest_normal * info.eps
        assert ((o.double() - want).abs() <= tol).all()
        assert out is None or torch.equal(b, g)
    return norm


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9, math.inf])
@pytest.mark.parametrize("dt", KINDS + [torch.float32])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 8192, 8193, 100003])
def test_clip_one_tensor(n, dt, max_norm):
    check_clip(grads_of([n], [dt], seed=n), max_norm)
    g = grads_of([n], [dt], seed=n)
    check_clip(g, max_norm, scale=0.25, out=[torch.empty_like(t) for t in g])


@pytest.mark.parametrize("count", [2, 64, 65, 300, 960, 961, 2000])
def test_clip_many_tensors(count):
    sizes = [(i * 7919 % 5000) + (i % 3 == 0) for i in range(count)]  # some hold nothing
    dts = [(KINDS + [torch.float32])[i % 3] for i in range(count)]
    check_clip(grads_of(sizes, dts, seed=count, size=0.01), 1.0, scale=0.5)
    g = grads_of(sizes, dts, seed=count, size=0.01)
    a = sf.clip_grad_norm(g, 1.0, out=[torch.empty_like(t) for t in g])
    assert torch.equal(a, sf.clip_grad_norm(g, 1.0, out=[torch.empty_like(t) for t in g]))  # one order of sums


@pytest.mark.parametrize("dt", KINDS + [torch.float32])
def test_clip_views_at_every_alignment(dt):
    buf = torch.randn(40000, device="cuda").to(dt)
    cuts = [1 + 37 * i for i in range(24)] + [30001]
    views = [buf[a:b] for a, b in zip(cuts, cuts[1:])]
    edge = buf[0].clone(), buf[30001:].clone()
    check_clip(views, 0.3)
    assert torch.equal(buf[0], edge[0]) and torch.equal(buf[30001:], edge[1])
    other = torch.empty(40000, device="cuda", dtype=dt)
    check_clip(views, 0.3, out=[other[3 + a:3 + b] for a, b in zip(cuts, cuts[1:])])


def test_clip_other_orders_of_dimensions():
    w = torch.randn(300, 40, device="cuda").half()
    g = [w.t(), torch.randn(3, 5, 7, device="cuda").permute(2, 0, 1), torch.randn((), device="cuda")]
    check_clip(g, 0.5)
    with pytest.raises(ValueError):
        sf.clip_grad_norm([torch.zeros(4, 8, device="cuda")[:, :7]], 1.0)
    with pytest.raises(ValueError):
        sf.clip_grad_norm([torch.zeros(1, device="cuda").expand(5)], 1.0)


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-12, 1e12, 1e19, 1e30])
def test_clip_ends_of_the_range(size):
    """Squares that leave fp32's range either way; the norm does not."""
    for dt in (torch.float32, torch.bfloat16):
        check_clip(grads_of([1000, 33], [dt, dt], size=size), size)
        mixed = grads_of([100], [dt], size=size) + grads_of([100], [dt], size=size * 1e-3)
        check_clip(mixed, 1e3 * size)


def test_clip_values_that_are_not_finite():
    g = grads_of([100, 50], [torch.float16, torch.float32])
    g[0][7] = float("inf")
    n = sf.clip_grad_norm(g, 1.0)
    assert n.item() == math.inf and g[0][7].isnan() and (g[0][:7] == 0).all() and (g[1] == 0).all()
    g = grads_of([100, 50], [torch.float16, torch.float32])
    g[1][3] = float("nan")
    n = sf.clip_grad_norm(g, 1.0)
    assert math.isnan(n.item()) and all(t.isnan().all() for t in g)
    z = [torch.zeros(1000, device="cuda"), torch.zeros(0, device="cuda")]
    assert sf.clip_grad_norm(z, 0.0).item() == 0 and (z[0] == 0).all()
    z = [torch.zeros(0, device="cuda")]
    assert sf.clip_grad_norm(z, 1.0).item() == 0


def test_clip_refuses_tensors_that_overlap():
    buf = torch.ones(100, device="cuda")
    for pair in ([buf, buf], [buf[:60], buf[50:]]):
        with pytest.raises(sf.SfnnError):
            sf.clip_grad_norm(pair, 1.0)
    with pytest.raises(sf.SfnnError):
        sf.clip_grad_norm([buf[:50]], 1.0, out=[buf[10:60]])
    with pytest.raises(sf.SfnnError):  # an output that is another gradient
        sf.clip_grad_norm([buf[:50], buf[50:]], 1.0, out=[buf[50:], buf[:50]])
    assert (buf == 1).all()
    out = [torch.empty(100, device="cuda") for _ in range(2)]
    sf.clip_grad_norm([buf, buf], 1.0, out=out)  # counted twice, read twice
    assert torch.equal(out[0], out[1])


def test_clip_in_a_graph_and_on_another_stream():
    g = grads_of([5000, 77], [torch.bfloat16, torch.float32])
    out = [torch.empty_like(t) for t in g]
    sf.clip_grad_norm(g, 1.0, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = sf.clip_grad_norm(g, 1.0, out=out)
    for size in (0.001, 3.0):
        for t in g:
            t.mul_(size)
        graph.replay()
        got = [norm.clone()] + [t.clone() for t in out]
        n = sf.clip_grad_norm(g, 1.0, out=out)
        for u, v in zip(got, [n] + out):
            assert torch.equal(u, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = [torch.empty_like(t) for t in g]
    n2 = sf.clip_grad_norm(g, 1.0, out=other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(n, n2) and all(torch.equal(u, v) for u, v in zip(out, other))


def test_out_that_shares_memory():
    d = 64
    buf = torch.randn(9, 3 * d, device="cuda").half()
    x, z, w = buf[:8, :d], buf[:8, d:2 * d], torch.ones(d, device="cuda").half()
    want = sf.residual_norm_forward(x, z, "rms", w)
    beside = sf.residual_norm_forward(x, z, "rms", w, out=buf[:8, 2 * d:])  # between the rows of x and z
    assert torch.equal(want[0], beside[0]) and torch.equal(want[1], beside[1])
    for out in (z, buf[1:, :d], buf[:8, 8:d + 8], buf[:8, d - 8:2 * d - 8]):
        with pytest.raises(ValueError, match="overlap"):
            sf.residual_norm_forward(x, z, "rms", w, out=out)
    with pytest.raises(ValueError, match="overlap"):
        sf.residual_norm_forward(x[:1], z[:1], "rms", w, out=w[None])
    inside = sf.residual_norm_forward(x, z, "rms", w, out=x)
    assert torch.equal(want[0], inside[0]) and torch.equal(want[1], inside[1])


# Neither a post norm nor a gate: the backward kernel without Z's own sums, its widths and what may be missing.
@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("pre", ["rms", "layer"])
@pytest.mark.parametrize("T,d", [(1, 512), (3, 8), (700, 512), (301, 1001), (150, 4096), (9, 4104), (40, 8192), (5, 8200), (3000, 96)])
def test_plain_branches(T, d, pre, dt):
    for i in range(3):
        check(T, d, dt, A=[1.0, 0.75, 1.0][i], C=[1.0, -0.5, 2.0][i], seed=T + i, pre=pre, bias=i != 1, x32=i == 1, z32=i == 2)
    a, rows, saved = check(T, d, dt, seed=d, pre=pre, bias=True, pad=i)
    dr, dh = rows(a["x"].dtype), rows(dt)
    full = sf.residual_norm_backward(dr, dh, saved)
    for j, k in enumerate(GRADS):  # one at a time
        one = sf.residual_norm_backward(dr, dh, saved, need=[i == j for i in range(7)])
        assert all((t is None) == (i != j or full[i] is None) for i, t in enumerate(one))
        if full[j] is not None:
            assert torch.equal(one[j], full[j]) if full[j].dim() == 2 else True
            near(one[j], *plain(a, pre, "none", 1.0, 1.0, dr, dh)[k], K=T if full[j].dim() == 1 else 0)
    for r_, h_ in ((dr, None), (None, dh)):  # one of the two is missing
        want = plain(a, pre, "none", 1.0, 1.0, torch.zeros_like(dr) if r_ is None else r_, h_)
        for k, v in zip(GRADS, sf.residual_norm_backward(r_, h_, saved)):
            if v is not None:
                near(v, *want.get(k, (torch.zeros_like(v, dtype=torch.float64),) * 2), K=T if v.dim() == 1 else 0)
