"""The dense operators used together: a small stack trained with 8-bit saved activations,
its weights then served as prompts through sparse-layer handles and as MXFP4 linears.  What
is checked is that it runs and that its gradients and outputs are the formulas'."""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu

D, N, LAYERS = 128, 320, 2


def make(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return [[(r(N, D) / D ** 0.5).half(), (r(N, D) / D ** 0.5).half(), (r(D, N) / N ** 0.5).half(),
             (0.1 * r(N) - 0.5).half()] for _ in range(LAYERS)], r


def forward(x, layers, checkpoint):
    for wg, wu, wd, b in layers:
        x = x + sf.gated_ffn(x, wg, wu, wd, b, checkpoint=checkpoint)
    return x


@pytest.mark.parametrize("checkpoint", ["full", "act8"])
def test_training_steps_run_and_give_the_formulas_gradients(checkpoint):
    layers, r = make(1)
    leaves = [[t.requires_grad_() for t in l] for l in layers]
    flat = [t for l in leaves for t in l]
    x, target = r(3, 41, D).half(), r(3, 41, D).half()
    for step in range(3):
        y = forward(x, leaves, checkpoint)
        grads = torch.autograd.grad(y, flat, ((y - target) / 8).detach())
        if step == 0:
            # the same stack in 64 bits; a gradient's error grows by each rounding on its way:
            # H, the residual, dU / dG and the result for each of the two layers, and an 8-bit
            # step of X, U and relu(G) (1/127 of a block's largest, about 3 of its deviations)
            p = [[t.detach().double().requires_grad_() for t in l] for l in layers]
            z = x.double()
            for wg, wu, wd, b in p:
                h = (z @ wg.t() + b).clamp_min(0) * (z @ wu.t())
                z = z + h @ wd.t()
            want = torch.autograd.grad(z, [t for l in p for t in l], ((y - target) / 8).detach().double())
            # in norm: roundings of 2^-11 a stage, twelve stages; act8's half step is
            # 3.5 / 127 / sqrt(12) of a deviation for each of two saved factors, plus the masks of
            # gates within fp16 rounding of zero (a share of 2^-9 of the active ones at most)
            bound = 12 * 2.0 ** -11 + 2 * 2.0 ** -4.5 * 2.0 ** -2 * (checkpoint == "act8") + 2.0 ** -4.5 * 0.2
            for a, w in zip(grads, want):
                assert torch.isfinite(a).all()
                assert (a.double() - w).norm() <= bound * w.norm()
        with torch.no_grad():
            for t, g in zip(flat, grads):
                t.sub_(0.01 * g)
    assert sf.dense_error() == 0


def test_trained_weights_serve_prompts_and_four_bits():
    layers, r = make(2)
    wg, wu, wd, b = layers[0]
    x = r(37, D).half()
    dense = sf.gated_ffn_forward(x, wg, wu, wd, b)[0]
    # the same layer behind a handle: prompts through its own rows, single tokens through its set
    A, B = (r(D, 32) / D ** 0.5).half(), (r(32, N) / 32 ** 0.5).half()
    h = sf.SparseFFN(wu, wd, b, A, B, torch.ones(N, device="cuda").half(), act="reglu", w_gate=wg, max_batch=8)
    prompt = h.forward_prompt(x)
    assert ((prompt.double() - dense.double()).abs() <= 2.0 ** -9 * dense.double().abs().clamp_min(0.25)).all()
    Y, idx, counts = h.forward_batch(x[:8], return_sets=True)
    assert torch.isfinite(Y).all() and h.get_error() == 0
    h.close()
    # 4-bit weights: each linear against the product of the values that the codes stand for
    qg, qu, qd = (sf.quantize_mxfp4(w) for w in (wg, wu, wd))
    gate, up = sf.mxfp4_linear(x, qg), sf.mxfp4_linear(x, qu)
    xv = sf.dequantize_mxfp4(sf.quantize_mxfp4(x)).double()
    for got, q in ((gate, qg), (up, qu)):
        want = xv @ sf.dequantize_mxfp4(q).double().t()
        assert ((got.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -14).all()
    hid = (gate + b).clamp_min(0) * up
    y4 = sf.mxfp4_linear(hid, qd)
    hv = sf.dequantize_mxfp4(sf.quantize_mxfp4(hid)).double()
    want = hv @ sf.dequantize_mxfp4(qd).double().t()
    assert ((y4.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -14).all()
    # its saved activations in 8 bits take about half of the 16-bit blocks
    _, full = sf.gated_ffn_forward(x, wg, wu, wd, b, save="full")
    _, eight = sf.gated_ffn_forward(x, wg, wu, wd, b, save="act8")
    assert eight.nbytes < 0.6 * full.nbytes
    assert sf.dense_error() == 0


def test_whole_step_in_one_graph_with_eager_calls_between():
    """Explicit forward and backward calls captured together and replayed on new inputs."""
    layers, r = make(3)
    wg, wu, wd, b = layers[0]
    x, dy = r(64, D).half(), r(64, D).half()

    def step():
        y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save="act8")
        grads = sf.gated_ffn_backward(dy, saved, wg, wu, wd)
        q = sf.quantize_mxfp4(wg)
        return [y, *grads, sf.mxfp4_linear(x, q), sf.dequantize_act8(sf.quantize_act8(y))]

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (5, 6):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(64, D, generator=gen, device="cuda"))
        dy.copy_(torch.randn(64, D, generator=gen, device="cuda"))
        wg.mul_(1.25)
        g.replay()
        got = [t.clone() for t in out]
        for a, w in zip(got, step()):
            assert torch.equal(a, w)
    assert sf.dense_error() == 0
