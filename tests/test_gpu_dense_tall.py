"""Products in tiles of 512 rows: a prompt's down projection in fp32, and that a row's results do not
depend on how many rows come with it (the sums run over K in one order in every tile)."""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,T", [(1024, 5001), (1000, 4700)])
def test_prompt_through_a_handle(d, T):
    import workload as W
    cfg = W.small_config(W.CONFIGS["opt6.7b_relu"], d=d, n=1000, r=64)
    lay = W.make_layer(cfg, seed=3)
    h = sf.SparseFFN.from_layer(lay, max_batch=2, device="cuda:0")
    X = torch.randn(T, d, generator=torch.Generator().manual_seed(T)).half().cuda()
    Y = h.forward_prompt(X)
    assert Y.dtype == torch.float32
    parts = [h.forward_prompt(X[i:i + 700]) for i in range(0, T, 700)]  # few rows: square tiles
    # a part's K may be split: twice the error of sums of n terms
    x, wu, wd, b = X.double(), *(torch.from_numpy(a).cuda().double() for a in (lay.w_up, lay.w_down, lay.b))
    H = (x @ wu.t() + b).clamp_min(0).half().double()
    tol = 2 * 1000 * 2.0 ** -23 * (H @ wd.abs().t()) + 2.0 ** -11 * 2.0 ** -24 * wd.abs().sum(1)
    off = (torch.cat(parts).double() - Y.double()).abs()
    assert (off <= tol + 2.0 ** -24 * Y.abs()).all()
    assert h.get_error() == 0
    h.close()


@pytest.mark.parametrize("T,K,N", [(5000, 1000, 2600), (4999, 1160, 2311)])
def test_rows_do_not_depend_on_one_another(T, K, N):
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    x, w, dy = r(T, K), r(N, K), r(T, N)
    _, saved = sf.linear_forward(x, w, None, "silu", save=True)
    dx, dw, _ = sf.linear_backward(dy, saved, w)
    assert torch.equal(dx, sf.linear_backward(dy, saved, w, need=(True, False, False))[0])
    assert torch.equal(dw, sf.linear_backward(dy, saved, w, need=(False, True, False))[1])
    for lo, hi in ((0, 2500), (2500, T)):
        _, part = sf.linear_forward(x[lo:hi], w, None, "silu", save=True)
        assert torch.equal(dx[lo:hi], sf.linear_backward(dy[lo:hi], part, w, need=(True, False, False))[0])


def test_two_streams_and_graphs():
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").half()
    x, w, b, dy = r(2500, 1000), r(2600, 1000) * 0.03, r(2600), r(2500, 2600)

    def step():
        y, saved = sf.linear_forward(x, w, b, "gelu", save=True)
        return (y, *sf.linear_backward(dy, saved, w), sf.linear_forward(x[:300], w, b, "relu")[0], sf.linear_forward(x[:7], w, b)[0])

    want = step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(step())
        graph.replay()
    torch.cuda.synchronize()
    for out in outs + [held]:
        assert all(torch.equal(a, c) for a, c in zip(out, want))
    assert sf.dense_error() == 0
