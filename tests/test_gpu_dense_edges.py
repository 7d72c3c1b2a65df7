"""The dense operators where they can go wrong at the edges: blocks that are not finite,
neurons of unlike size, values at the ends of the range, streams, saved memory, counters.
Tolerances count half a step of the type (eps / 2) per rounding."""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf
from test_gpu_dense import KINDS, layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("save", ["full", "act8"])
@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("where", ["w_gate", "b", "x", "w_up"])
def test_gradients_of_blocks_that_are_not_finite(where, T, save, dt):
    """A block of 64 neurons whose gate holds a NaN or an infinity gives NaN gradients, as the
    formula does; the other blocks (for a token: the other tokens) keep theirs to the bit."""
    x, wg, wu, wd, b, dy = layer(T, 72, 200, dt, seed=T)
    y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save=save)
    want = sf.gated_ffn_backward(dy, saved, wg, wu, wd)
    on = (x.double() @ wg.double().t() + b.double()) > 0
    x2, wg2, wu2, b2 = x.clone(), wg.clone(), wu.clone(), b.clone()
    block = torch.zeros(200, dtype=torch.bool, device="cuda")
    block[64:128] = True
    if where == "w_gate":
        wg2[70, 3] = float("nan")
    elif where == "b":
        b2[70] = float("inf")
    elif where == "x":
        x2[2, 3] = float("nan")
    else:
        wu2[70, 3] = float("nan")
    y, saved = sf.gated_ffn_forward(x2, wg2, wu2, wd, b2, save=save)
    dx, dwg, dwu, dwd, db = sf.gated_ffn_backward(dy, saved, wg, wu, wd)
    if where == "x":  # one token: in every neuron's sum, and in its own row of dX
        rest = torch.arange(T, device="cuda") != 2
        assert dx[2].isnan().all() and torch.equal(dx[rest], want[0][rest])
        for g in (dwg, dwu, dwd, db):
            assert g.isnan().all()
    elif where == "w_up":  # U's block: dG of the neurons that are on, and H; dU = dH relu(G) does not read it
        hit = block & on.any(0)
        assert db[hit].isnan().all() and dwg[hit].isnan().all() and dwd[:, block].isnan().all()
        assert (db[block & ~hit] == 0).all() and (dwg[block & ~hit] == 0).all()
        assert torch.equal(dwu, want[2])
    else:
        assert db[block].isnan().all() and dwg[block].isnan().all() and dwu[block].isnan().all()
        assert dwd[:, block].isnan().all() and dx.isnan().all()
    if where != "x":
        for g, w in ((db, want[4]), (dwg, want[1]), (dwu, want[2]), (dwd.t(), want[3].t())):
            assert torch.equal(g[~block], w[~block])
    assert sf.dense_error() == 0
