"""linear, residual_norm and their plain calls under forward mode and torch.func's transforms: refused where a
tangent, a gradient or a batch dimension would be lost, else as without them."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu


def normal(*shape, seed=0, dt=torch.float16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def linear_args():
    return [normal(6, 64), normal(40, 64, seed=1), normal(40, seed=2), normal(6, 40, seed=3)]


def norm_args():
    return [normal(6, 64), normal(6, 64, seed=1), normal(64, seed=2), normal(64, seed=3), normal(64, seed=4), normal(64, seed=5),
            normal(64, seed=6)]


def linear(x, w, b, res):
    return sf.linear(x, w, b, "gelu", res)


def norm(x, z, w, b, post_w, post_b, gate):
    return sf.residual_norm(x, z, "layer", w, b, "rms", post_w, post_b, gate)[1]


def norm_alone(x, *rest):
    return sf.residual_norm(x, None, "rms", rest[1])[1]


OPS = [(linear, linear_args), (norm, norm_args), (norm_alone, norm_args)]
USED = {linear: range(4), norm: range(7), norm_alone: (0, 2)}


@pytest.mark.parametrize("op,make", OPS)
def test_forward_mode_is_refused(op, make):
    args = make()
    want = op(*args)
    with fw.dual_level():
        for i in USED[op]:
            dual = [fw.make_dual(t, torch.ones_like(t)) if j == i else t for j, t in enumerate(args)]
            with pytest.raises((RuntimeError, NotImplementedError)):
                op(*dual)
        assert torch.equal(op(*args), want)  # no tangent: nothing to refuse
    assert torch.equal(op(*args), want)
    for i in USED[op]:
        with pytest.raises((RuntimeError, NotImplementedError)):
            torch.func.jvp(lambda t: op(*args[:i], t, *args[i + 1:]), (args[i],), (torch.ones_like(args[i]),))


@pytest.mark.parametrize("op,make", OPS)
def test_gradients_and_batches_of_functions_are_refused(op, make):
    args = make()
    for i in USED[op]:
        def of_one(t):
            return op(*args[:i], t, *args[i + 1:])
        with pytest.raises((RuntimeError, NotImplementedError)):
            torch.func.grad(lambda t: of_one(t).float().sum())(args[i])
        with pytest.raises((RuntimeError, NotImplementedError)):
            torch.func.vmap(of_one)(torch.stack([args[i]] * 2))


def test_plain_calls_of_batches_are_refused():
    x, w, b, res = linear_args()
    two = lambda t: torch.stack([t, t])
    y, saved = sf.linear_forward(x, w, b, "relu", save=True)
    r, h, kept = sf.residual_norm_forward(x, x, save=True)
    for f, t in ((lambda t: sf.linear_forward(t, w, b)[0], x), (lambda t: sf.linear_forward(x, w, t)[0], b),
                 (lambda t: sf.linear_forward(x, w, b, residual=t)[0], res), (lambda t: sf.linear_backward(t, saved, w)[0], y),
                 (lambda t: sf.residual_norm_forward(t, x)[0], x), (lambda t: sf.residual_norm_forward(x, t)[0], x),
                 (lambda t: sf.residual_norm_backward(t, None, kept)[0], r), (lambda t: sf.clip_grad_norm([t], 1.0), y)):
        with pytest.raises((RuntimeError, NotImplementedError, TypeError, ValueError)):
            torch.func.vmap(f)(two(t))
    assert sf.dense_error() == 0


def test_tensors_whose_memory_is_not_their_values():
    """Negated when read (the imaginary part of a conjugate), or not in rows at all: refused, also where an optional
    argument is one."""
    parts = torch.view_as_complex(torch.randn(6, 40, 2, device="cuda"))
    neg = parts.conj().imag
    assert neg.is_neg() and not neg.resolve_neg().is_neg()
    x, w, b, _ = linear_args()
    sparse = torch.eye(40, device="cuda").to_sparse()
    rows, sparse_rows = neg.resolve_neg().contiguous(), torch.randn(6, 40, device="cuda").to_sparse()
    for bad in (neg, sparse_rows):
        for call in (lambda: sf.linear_forward(x, w, b, residual=bad), lambda: sf.linear_forward(x, w, b, out=bad, out_dtype=torch.float32),
                     lambda: sf.residual_norm_forward(bad, rows, dtype=torch.float16), lambda: sf.clip_grad_norm([bad], 1.0),
                     lambda: sf.residual_norm_forward(rows, bad, dtype=torch.float16), lambda: sf.clip_grad_norm([rows], 1.0, out=[bad])):
            with pytest.raises(TypeError):
                call()
    with pytest.raises(TypeError):
        sf.linear_forward(x, w, sparse[0].half())
    assert sf.linear_forward(x, w, b, residual=rows)[0].shape == (6, 40) and sf.dense_error() == 0
