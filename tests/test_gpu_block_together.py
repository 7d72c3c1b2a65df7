"""The operators around the products used together: an OPT-shaped stack (LayerNorm, linear with ReLU,
linear onto an fp32 residual) trained for a step and clipped, a gated block between its two norms,
and decode steps of sparse layers joined by norms.  What is checked is that it runs and that its
gradients and outputs are the formulas'."""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu

D, N, LAYERS, EPS = 128, 328, 2, 1e-5


def make(seed, dt):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return [[(1 + 0.1 * r(D)).to(dt), (0.1 * r(D)).to(dt), (r(N, D) / D ** 0.5).to(dt), (0.1 * r(N)).to(dt),
             (r(D, N) / N ** 0.5).to(dt), (0.1 * r(D)).to(dt)] for _ in range(LAYERS)], r


def stack(x, layers):
    """The residual stream (fp32) through the layers: h = LayerNorm(x), x + W2 relu(W1 h + b1) + b2."""
    for w, b, w1, b1, w2, b2 in layers:
        _, h = sf.residual_norm(x, pre="layer", w=w, b=b, eps=EPS)
        x = sf.linear(sf.linear(h, w1, b1, act="relu"), w2, b2, residual=x)
    return x


def stack64(x, layers):
    for w, b, w1, b1, w2, b2 in layers:
        c = x - x.mean(-1, keepdim=True)
        h = c / (c.square().mean(-1, keepdim=True) + EPS).sqrt() * w + b
        x = x + (h @ w1.t() + b1).clamp_min(0) @ w2.t() + b2
    return x


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_a_training_step_and_its_clipping(dt):
    layers, r = make(1, dt)
    flat = [t.requires_grad_() for l in layers for t in l]
    x = r(3, 41, D).requires_grad_()
    dy = r(3, 41, D)
    y = stack(x, layers)
    assert y.dtype == torch.float32 and y.shape == x.shape
    grads = torch.autograd.grad(y, [x] + flat, dy)
    p = [[t.detach().double().requires_grad_() for t in l] for l in layers]
    z = x.detach().double().requires_grad_()
    want = torch.autograd.grad(stack64(z, p), [z] + [t for l in p for t in l], dy.double())
    # in norm: h, the hidden layer, dZ of both products and the result are rounded (eps / 2 each) in both
    # layers, ten roundings on the longest way; a ReLU decided otherwise within the rounding of its input
    # (a share of eps of the values, each worth at most its whole term)
    half = torch.finfo(dt).eps / 2
    bound = 10 * half + (2 * half) ** 0.5 * 0.5
    for a, w in zip(grads, want):
        assert torch.isfinite(a).all()
        assert (a.double() - w).norm() <= bound * w.norm()
    # one norm over all of them, in place
    before = [g.clone() for g in grads[1:]]
    total = torch.stack([g.double().square().sum() for g in before]).sum().sqrt().item()
    norm = sf.clip_grad_norm(list(grads[1:]), 0.5 * total)
    assert abs(norm.item() - total) <= 2.0 ** -20 * total
    for g, b in zip(grads[1:], before):
        assert ((g.double() - 0.5 * b.double()).abs() <= (half + 2.0 ** -18) * 0.5 * b.double().abs() + 2.0 ** -25).all()
    after = torch.stack([g.double().square().sum() for g in grads[1:]]).sum().sqrt().item()
    assert abs(after - 0.5 * total) <= (half + 2.0 ** -18) * total
    assert sf.dense_error() == 0


def test_a_gated_block_between_its_norms():
    """r = x + gate * RMS(gated_ffn(RMS(x))): pre and post norm around the framework's own block."""
    dt = torch.bfloat16
    _, r = make(2, dt)
    wg, wu, wd = (r(N, D) / D ** 0.5).to(dt), (r(N, D) / D ** 0.5).to(dt), (r(D, N) / N ** 0.5).to(dt)
    w1, w2, w3, gate = ((1 + 0.1 * r(D)).to(dt) for _ in range(4))
    x = r(50, D).to(dt)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu, wd, w1, w2, w3, gate)]
    x_, wg_, wu_, wd_, w1_, w2_, w3_, gate_ = leaves
    _, h = sf.residual_norm(x_, w=w1_, eps=EPS)
    y = sf.gated_ffn(h, wg_, wu_, wd_)
    res, out = sf.residual_norm(x_, y, "rms", w3_, post="rms", post_w=w2_, gate=gate_, eps=EPS)
    dr, dh = r(50, D).to(dt), r(50, D).to(dt)
    got = torch.autograd.grad([res, out], leaves, [dr, dh])

    def rms(v):
        return v / (v.square().mean(-1, keepdim=True) + EPS).sqrt()
    p = [t.detach().double().requires_grad_() for t in leaves]
    X, WG, WU, WD, W1, W2, W3, G = p
    H = rms(X) * W1
    Y = ((H @ WG.t()).clamp_min(0) * (H @ WU.t())) @ WD.t()
    R = X + G * (rms(Y) * W2)
    want = torch.autograd.grad([R, rms(R) * W3], p, [dr.double(), dh.double()])
    half = torch.finfo(dt).eps / 2
    for a, w in zip(got, want):  # roundings of h, H, y, dy, dG, dU and the result, and gates near zero as above
        assert (a.double() - w).norm() <= (9 * half + (2 * half) ** 0.5 * 0.5) * w.norm()
    assert sf.dense_error() == 0


def test_decode_steps_joined_by_norms():
    """Two sparse layers decode a token: the first's fp32 output joins the fp32 residual, its norm is the
    second's input; then a linear layer onto the residual, in place."""
    _, r = make(3, torch.float16)
    handles = []
    for _ in range(2):
        w = [(r(N, D) / D ** 0.5).half(), (r(D, N) / N ** 0.5).half(), (0.1 * r(N)).half(), (r(D, 32) / D ** 0.5).half(),
             (r(32, N) / 32 ** 0.5).half(), torch.ones(N, device="cuda").half()]
        handles.append(sf.SparseFFN(*w, act="relu"))
    norm_w = (1 + 0.1 * r(D)).half()
    x = r(D)
    _, h, _ = sf.residual_norm_forward(x, w=norm_w, eps=EPS)
    y = handles[0].forward(h)
    want = x + y
    out, h2, _ = sf.residual_norm_forward(x, y, w=norm_w, eps=EPS, out=x)
    assert out is x and torch.equal(x, want)
    v = want.double()
    hw = v / (v.square().mean() + EPS).sqrt() * norm_w.double()
    assert ((h2.double() - hw).abs() <= (2.0 ** -11 + 2.0 ** -18) * hw.abs() + 2.0 ** -25).all()
    y2 = handles[1].forward(h2)
    w, b = (r(D, D) / D ** 0.5).half(), (0.1 * r(D)).half()
    res = x.view(1, D).clone()
    z, _ = sf.linear_forward(h2.view(1, D), w, b, "gelu", residual=res, out=res)
    Z = h2.double() @ w.double().t() + b.double()
    want = x.double() + Z * torch.special.ndtr(Z)
    # K products in 32 bits, the activation's 8 roundings, the sum's
    tol = 1.13 * D * 2.0 ** -23 * (h2.double().abs() @ w.double().abs().t() + b.double().abs()) + 2.0 ** -20 * Z.abs() + \
        2.0 ** -24 * want.abs()
    assert z is res and ((res.double()[0] - want).abs() <= 1.01 * tol).all()
    assert torch.isfinite(y2).all()
    for hd in handles:
        assert hd.get_error() == 0
        hd.close()
    assert sf.dense_error() == 0


def test_a_whole_step_in_one_graph():
    """Forward, backward and clipping as explicit calls, captured together and replayed on new inputs."""
    layers, r = make(4, torch.bfloat16)
    w, b, w1, b1, w2, b2 = layers[0]
    x, dy = r(64, D), r(64, D)

    def step():
        _, h, sn = sf.residual_norm_forward(x, None, "layer", w, b, eps=EPS, save=True)
        a, s1 = sf.linear_forward(h, w1, b1, "relu", save=True)
        y, s2 = sf.linear_forward(a, w2, b2, residual=x, save=True)
        da, dw2, db2 = sf.linear_backward(dy, s2, w2)
        dh, dw1, db1 = sf.linear_backward(da, s1, w1)
        dx, _, _, dw, db, _, _ = sf.residual_norm_backward(dy, dh, sn)
        grads = [dw, db, dw1, db1, dw2, db2]
        return [y, dx, sf.clip_grad_norm(grads, 1.0)] + grads
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (5, 6):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(64, D, generator=gen, device="cuda"))
        dy.copy_(torch.randn(64, D, generator=gen, device="cuda"))
        w1.mul_(1.25)
        g.replay()
        got = [t.clone() for t in out]
        for u, v in zip(got, step()):
            assert torch.equal(u, v)
    assert sf.dense_error() == 0
