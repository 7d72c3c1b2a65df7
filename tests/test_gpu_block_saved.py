"""What linear and residual_norm keep between their passes, where it comes back otherwise (saved-tensor
hooks that pack it, a caller that builds the saved object): refused before anything reads it."""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu


def normal(*shape, seed=0, dt=torch.float16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


OTHERWISE = [lambda t: t[:-1], lambda t: t.double(), lambda t: t.cpu(), lambda t: t.reshape(-1, 1), lambda t: torch.cat([t, t]),
             lambda t: t.repeat_interleave(2, 0)[::2]]


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("change", OTHERWISE)
def test_slopes(change, act):
    x, w, dy = normal(9, 64), normal(40, 64, seed=1), normal(9, 40, seed=2)
    leaf = w.clone().requires_grad_()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: change(t) if t.dtype == torch.uint8 else t):
        y = sf.linear(x, leaf, act=act)
    with pytest.raises(ValueError, match="slopes"):
        torch.autograd.grad(y, leaf, dy)
    _, saved = sf.linear_forward(x, w, act=act, save=True)
    for slopes in (None, change(saved.slopes)):
        with pytest.raises(ValueError, match="slopes"):
            sf.linear_backward(dy, sf.LinearSaved(x, slopes, saved.act, saved.N, saved.y_dtype, False), w)


@pytest.mark.parametrize("change", OTHERWISE)
def test_stats(change):
    x, z, dr = normal(9, 64), normal(9, 64, seed=1), normal(9, 64, seed=2)
    leaf = z.clone().requires_grad_()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: change(t) if t.dtype == torch.float32 else t):
        r, h = sf.residual_norm(x, leaf)
    with pytest.raises(ValueError, match="stats"):
        torch.autograd.grad(h, leaf, dr)
    _, _, saved = sf.residual_norm_forward(x, z, save=True)
    for stats in (None, change(saved.stats)):
        with pytest.raises(ValueError, match="stats"):
            sf.residual_norm_backward(dr, dr, sf.NormSaved(saved.tensors, stats, saved.options, saved.dtype))


def test_hooks_that_bring_everything_back():
    x, w, b, dy = normal(9, 64), normal(40, 64, seed=1), normal(40, seed=2), normal(9, 40, seed=3)
    _, saved = sf.linear_forward(x, w, b, "gelu", save=True)
    want = sf.linear_backward(dy, saved, w)
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    with torch.autograd.graph.save_on_cpu(pin_memory=True):
        y = sf.linear(*leaves, act="gelu")
    assert all(torch.equal(u, v) for u, v in zip(torch.autograd.grad(y, leaves, dy), want))
    z = normal(9, 64, seed=4)
    _, _, saved = sf.residual_norm_forward(x, z, "layer", save=True)
    want = sf.residual_norm_backward(x, z, saved)[:2]
    leaves = [t.clone().requires_grad_() for t in (x, z)]
    with torch.autograd.graph.save_on_cpu():
        r, h = sf.residual_norm(*leaves, pre="layer")
    assert all(torch.equal(u, v) for u, v in zip(torch.autograd.grad([r, h], leaves, [x, z]), want))
    # nothing is kept of no activation
    _, saved = sf.linear_forward(x, w, b, save=True)
    assert saved.slopes is None and sf.linear_backward(dy, saved, w)[1] is not None
    assert sf.dense_error() == 0
