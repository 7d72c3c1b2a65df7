"""What is written in place counts as changed: autograd refuses a backward pass that saved what was
there before, as it does after PyTorch's own operations in place."""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu


def normal(*shape, seed=0, dt=torch.float16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


def onto_residual(t):
    sf.linear_forward(normal(6, 64), normal(40, 64, seed=1), residual=t, out=t)


def into_rows(t):
    sf.linear_forward(normal(6, 64), normal(40, 64, seed=1), out=t)


def next_stream(t):
    sf.residual_norm_forward(t, normal(6, 40, seed=2), "rms", out=t)


def norm_into(t):
    sf.residual_norm_forward(normal(6, 40), normal(6, 40, seed=2), "rms", out=t)


def clipped(t):
    sf.clip_grad_norm([normal(5), t], 1e-3)


def clipped_into(t):
    sf.clip_grad_norm([normal(5), normal(6, 40)], 1.0, out=[torch.empty(5, device="cuda").half(), t])


def dequantized(t):
    sf.dequantize_act8(sf.quantize_act8(normal(6, 40, seed=7)), out=t)


WRITERS = [onto_residual, into_rows, next_stream, norm_into, clipped, clipped_into, dequantized]


@pytest.mark.parametrize("write", WRITERS)
def test_a_saved_tensor_that_is_overwritten_is_noticed(write):
    t = normal(6, 40, seed=3)
    leaf = normal(6, 40, seed=4).requires_grad_()
    y = (leaf * t).sum()  # saves t
    before = t._version
    write(t)
    assert t._version == before + 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("write", WRITERS)
def test_a_view_counts_for_its_buffer_and_inference_tensors_for_nothing(write):
    buf = normal(9, 48, seed=5)
    before = buf._version
    write(buf[1:7, :40]) if write not in (clipped, clipped_into) else write(buf.view(-1)[:240].view(6, 40))
    assert buf._version == before + 1
    with torch.inference_mode():
        inside = normal(6, 40, seed=6)
        write(inside)
    write(inside)  # outside the mode as well
    assert inside.is_inference()


def test_what_is_read_stays_as_it_is():
    """Inputs keep their count: a call that writes new tensors disturbs no backward pass."""
    x, w, z = normal(6, 64), normal(40, 64, seed=1), normal(6, 64, seed=2)
    grads = [normal(7, seed=3), normal(6, 40, seed=4)]
    before = [t._version for t in (x, w, z, *grads)]
    y, saved = sf.linear_forward(x, w, residual=None, save=True)
    sf.linear_backward(y, saved, w)
    r, h, saved = sf.residual_norm_forward(x, z, "rms", save=True)
    sf.residual_norm_backward(r, h, saved)
    sf.clip_grad_norm(grads, 1.0, out=[torch.empty_like(t) for t in grads])
    assert [t._version for t in (x, w, z, *grads)] == before
