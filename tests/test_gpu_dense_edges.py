"""The dense operators where they can go wrong at the edges: blocks that are not finite,
neurons of unlike size, values at the ends of the range, streams, saved memory, counters.
Tolerances count half a step of the type (eps / 2) per rounding."""
import pytest
import torch

import activation_sparse_ffn_threshold_b200 as sf
from test_gpu_dense import KINDS, backward64, forward64, layer, near

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


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("which", ["w_up", "w_gate"])
@pytest.mark.parametrize("T,d,n", [(1, 72, 264), (40, 264, 520), (300, 136, 1000)])
def test_full_gradients_of_neurons_of_unlike_size(T, d, n, which, dt):
    """Neurons that share a block with others up to 2^12 times as large keep their gradients'
    precision: a saved relu(G) is off by at most 2^-13 of itself and a saved U by 2^-12, or, far
    below the block's largest, either by 2^-23 of that."""
    x, wg, wu, wd, b, dy = layer(T, d, n, dt, seed=T + 1)
    dy = (dy.float() / 64).to(dt)  # (fp16's range)
    size = 0.25 * torch.tensor([1.0, 8.0, 64.0, 512.0, 4096.0], device="cuda")[torch.arange(n, device="cuda") * 7 % 5]
    if which == "w_up":
        wu = (wu.float() * size[:, None]).to(dt)
    else:  # (powers of two: the gate's sums stay exact)
        wg, b = (wg.float() * size[:, None]).to(dt), (b.float() * size).to(dt)
    y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save="full")
    got = sf.gated_ffn_backward(dy, saved, wg, wu, wd)
    G, U, H = forward64(x, wg, wu, wd, b)
    on = (G > 0).double()
    R = G * on
    want, terms = backward64(x, wg, wu, wd, dy, R, U, on)

    def top(v):
        v = torch.nn.functional.pad(v.abs(), (0, -n % 64)).view(T, -1, 64)
        return v.amax(2, keepdim=True).expand_as(v).reshape(T, -1)[:, :n]
    eR, eU = R * 2.0 ** -13 + top(R) * 2.0 ** -23, U.abs() * 2.0 ** -12 + top(U) * 2.0 ** -23
    # U is an fp32 sum besides: d 2^-23 of its terms
    eU = eU + d * 2.0 ** -23 * (x.double().abs() @ wu.double().abs().t())
    adH = dy.double().abs() @ wd.double().abs()
    eG, eV = adH * eU * on, adH * eR
    wg64, wu64, x64 = wg.double().abs(), wu.double().abs(), x.double().abs()
    extra = (eG @ wg64 + eV @ wu64, eG.t() @ x64, eV.t() @ x64, dy.double().abs().t() @ (eR * U.abs() + eU * R),
             eG.sum(0))
    for i, (g, K) in enumerate(zip(got, (2 * n + d, T + d, T + d, T + d, T + d))):
        if g is not None:
            near(g, want[i], terms[i] + extra[i] / (torch.finfo(dt).eps / 2), dt, 1, K)
    assert sf.dense_error() == 0


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("save", ["full", "act8"])
def test_bias_gradient_sums_what_was_not_rounded(save, dt):
    """Equal tokens round dG the same way, so a db that added up rounded values would carry that
    rounding whole; it adds the 32-bit ones and is rounded once."""
    T, d, n = 685, 64, 2048
    x, wg, wu, wd, b, dy = layer(1, d, n, dt, seed=5)
    x, dy = x.expand(T, d).contiguous(), dy.expand(T, d).contiguous()
    y, saved = sf.gated_ffn_forward(x, wg, wu, wd, b, save=save)
    db = sf.gated_ffn_backward(dy, saved, wg, wu, wd, need=(False, False, False, False, True))[4]
    G, U, H = forward64(x[:1], wg, wu, wd, b)
    on = (G > 0).double()
    if save == "full":  # U is an fp32 sum of d products, held to 2^-12 of itself or 2^-23 of its block's largest
        eU = d * 2.0 ** -23 * (x[:1].double().abs() @ wu.double().abs().t()) + 2.0 ** -12 * U.abs() + 2.0 ** -23 * U.abs().max()
    else:
        U = saved.u.view(torch.int8)[:1, :n].double() * saved.u_scales[:1].double().repeat_interleave(64, 1)[:, :n]
        eU = 2.0 ** -24 * U.abs()
    dH, adH = dy[:1].double() @ wd.double(), dy[:1].double().abs() @ wd.double().abs()
    want = T * dH * U * on
    # db's own rounding; U's error; dH is an fp32 sum of d products, db one of T
    tol = (torch.finfo(dt).eps / 2 + T * 2.0 ** -23) * want.abs() + T * on * (dH.abs() * eU + d * 2.0 ** -23 * adH * U.abs())
    assert ((db.double() - want[0]).abs() <= 1.001 * tol[0]).all()
    # the same sum where the other gradients' launch adds it up
    assert torch.equal(db, sf.gated_ffn_backward(dy, saved, wg, wu, wd)[4])
    assert sf.dense_error() == 0


@pytest.mark.parametrize("T", [1, 2, 3, 4, 6])
def test_mxfp4_scales_at_the_ends_of_the_range(T):
    """A block's sum of products times one scale may pass 2^128 where both scales bring it back."""
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    for kx, kw in ((2.0 ** 124, 2.0 ** -20), (2.0 ** -120, 2.0 ** 100), (2.0 ** -20, 2.0 ** 124)):
        x, w = (r(T, 288) * kx).to(torch.bfloat16), (r(100, 288) * kw).to(torch.bfloat16)
        q = sf.quantize_mxfp4(w)
        X, Wv = (sf.dequantize_mxfp4(v).double() for v in (sf.quantize_mxfp4(x), q))  # exact in bf16
        want, terms = X @ Wv.t(), X.abs() @ Wv.abs().t()
        got = sf.mxfp4_linear(x, q, out_dtype=torch.float32).double()
        assert ((got - want).abs() <= 2.0 ** -24 * want.abs() + 288 * 2.0 ** -23 * terms).all()
    assert sf.dense_error() == 0


def _handle(act, d, n, seed=3, **kw):
    import workload as W
    cfg = W.small_config(W.CONFIGS["70b_reglu" if act == "reglu" else "opt6.7b_relu"], d=d, n=n, r=64)
    return sf.SparseFFN.from_layer(W.make_layer(cfg, seed=seed), device="cuda:0", **kw)


def test_prompt_output_belongs_to_the_stream_that_writes_it():
    """Memory that the current stream freed may still be in use there: a call on another stream
    takes its output from that stream's own."""
    h = _handle("reglu", 128, 72)
    X = torch.randn(30001, 128, generator=torch.Generator().manual_seed(1)).half().cuda()
    want = h.forward_prompt(X)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.empty(30001, 128, device="cuda")
    at = old.data_ptr()
    old.fill_(7.0)
    del old
    Y = h.forward_prompt(X, stream=side)
    side.synchronize()
    assert Y.data_ptr() != at
    assert torch.equal(Y, want)
    h.close()


def test_prompt_workspace_is_sized_on_the_layers_device(monkeypatch):
    h = _handle("reglu", 128, 72)
    inside, sized = [], []

    class Device(torch.cuda.device):
        def __enter__(self):
            inside.append(self.idx)
            return super().__enter__()

        def __exit__(self, *a):
            inside.pop()
            return super().__exit__(*a)

    class Library:
        def __getattr__(self, name):
            if name == "sfnn_gated_workspace":
                sized.append(list(inside))
            return getattr(lib, name)
    lib, h._lib = h._lib, Library()
    monkeypatch.setattr(torch.cuda, "device", Device)
    X = torch.randn(3, 128, generator=torch.Generator().manual_seed(1)).half().cuda()
    h.forward_prompt(X, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert sized and all(0 in s for s in sized)
    monkeypatch.undo()
    h._lib = lib
    h.close()


@pytest.mark.parametrize("checkpoint", ["full", "act8"])
def test_saved_activations_end_with_the_backward_pass(checkpoint):
    x, wg, wu, wd, b, dy = layer(512, 256, 2048, torch.bfloat16, seed=6)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu, wd, b)]
    want = sf.gated_ffn_backward(dy, sf.gated_ffn_forward(x, wg, wu, wd, b, save=checkpoint)[1], wg, wu, wd)
    torch.cuda.synchronize()
    bare = torch.cuda.memory_allocated()
    y = sf.gated_ffn(*leaves, checkpoint=checkpoint)
    held = torch.cuda.memory_allocated() - bare - y.numel() * y.element_size()
    assert held >= 2 * 512 * 2048 * (2 if checkpoint == "full" else 1)
    for again in (True, False):
        grads = torch.autograd.grad(y, leaves, dy, retain_graph=again)
        assert all(torch.equal(a, c) for a, c in zip(grads, want))
        del grads
        left = torch.cuda.memory_allocated() - bare - y.numel() * y.element_size()
        assert left == held if again else left <= 0, "y is still here, what its backward pass read is not"
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, leaves, dy)


@pytest.mark.parametrize("checkpoint", ["full", "act8"])
def test_saved_activations_pass_through_hooks(checkpoint):
    """As every tensor that autograd saves: offloaded, and back at other addresses."""
    x, wg, wu, wd, b, dy = layer(100, 64, 200, torch.float16, seed=7)
    leaves = [t.clone().requires_grad_() for t in (x, wg, wu, wd, b)]
    want = sf.gated_ffn_backward(dy, sf.gated_ffn_forward(x, wg, wu, wd, b, save=checkpoint)[1], wg, wu, wd)
    packed = []

    def pack(t):
        packed.append(t.numel() * t.element_size())
        return t.cpu()
    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t.cuda()):
        y = sf.gated_ffn(*leaves, checkpoint=checkpoint)
    assert max(packed) >= 2 * 100 * 200 * (2 if checkpoint == "full" else 1)
    junk = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")  # over what the forward pass freed
    grads = torch.autograd.grad(y, leaves, dy)
    assert all(torch.equal(a, c) for a, c in zip(grads, want))
    del junk


def test_saved_activations_that_come_back_otherwise_are_refused():
    x, wg, wu, wd, b, dy = layer(10, 64, 128, torch.float16, seed=7)
    leaf = wg.clone().requires_grad_()
    for unpack in (lambda t: t[:-16] if t.dtype == torch.uint8 else t, lambda t: t.int() if t.dtype == torch.uint8 else t,
                   lambda t: t.cpu() if t.dtype == torch.uint8 else t):
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
            y = sf.gated_ffn(x, leaf, wu, wd, b)
        with pytest.raises(ValueError):
            torch.autograd.grad(y, leaf, dy)


def test_forward_mode_is_refused():
    import torch.autograd.forward_ad as fw
    x, wg, wu, wd, b, dy = layer(8, 64, 128, torch.float16, seed=8)
    want = sf.gated_ffn(x, wg, wu, wd, b)
    with fw.dual_level():
        for i in (0, 1, 4):
            args = [x, wg, wu, wd, b]
            args[i] = fw.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises((RuntimeError, NotImplementedError)):
                sf.gated_ffn(*args)
        assert torch.equal(sf.gated_ffn(x, wg, wu, wd, b), want)  # no tangent: nothing to refuse
    assert torch.equal(sf.gated_ffn(x, wg, wu, wd, b), want)


@pytest.mark.parametrize("T", [2, 40])
def test_mxfp4_linear_says_that_it_has_no_gradient(T):
    import torch.autograd.forward_ad as fw
    x, wg, *_ = layer(T, 64, 128, torch.float16, seed=9)
    q = sf.quantize_mxfp4(wg)
    want = sf.mxfp4_linear(x, q)
    leaf = x.clone().requires_grad_()
    y = sf.mxfp4_linear(leaf * 1, q)
    assert torch.equal(y, want)
    with pytest.raises(RuntimeError, match="gradient"):
        y.sum().backward()
    with torch.no_grad():
        y = sf.mxfp4_linear(leaf, q)
    assert not y.requires_grad and torch.equal(y, want)
    with fw.dual_level(), pytest.raises((RuntimeError, NotImplementedError)):
        sf.mxfp4_linear(fw.make_dual(x, torch.ones_like(x)), q)


@pytest.mark.parametrize("act", ["reglu", "relu"])
@pytest.mark.parametrize("d,n,T,kernels", [(512, 2051, 33, 3), (512, 2051, 300, 3), (128, 72, 33, 2), (128, 72, 1, 2)])
def test_prompt_counts_its_launches(d, n, T, kernels, act):
    """A down product whose K is split (few tiles, many neurons) joins its parts in a kernel of its own."""
    h = _handle(act, d, n)
    X = torch.randn(T, d, generator=torch.Generator().manual_seed(1)).half().cuda()
    before = h.info()["launches"]
    h.forward_prompt(X)
    assert h.info()["launches"] - before == kernels
    h.close()


@pytest.mark.parametrize("rows", [1, 2, 3, 4])
def test_mxfp4_blocks_that_are_not_finite_with_few_tokens(rows):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, 160, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(96, 160, generator=g, device="cuda").to(torch.bfloat16)
    q = sf.quantize_mxfp4(w)
    want = sf.mxfp4_linear(x, q)
    for bad in (float("nan"), float("inf"), float("-inf")):
        for t in range(rows):  # one token's block: its whole output, no other token's
            x2 = x.clone()
            x2[t, 70] = bad
            got = sf.mxfp4_linear(x2, q)
            rest = torch.arange(rows, device="cuda") != t
            assert got[t].isnan().all() and torch.equal(got[rest], want[rest])
        w2 = w.clone()  # one weight row's block: its column
        w2[5, 130] = bad
        got = sf.mxfp4_linear(x, sf.quantize_mxfp4(w2))
        keep = torch.arange(96, device="cuda") != 5
        assert got[:, 5].isnan().all() and torch.equal(got[:, keep], want[:, keep])
    assert sf.dense_error() == 0


@pytest.mark.parametrize("dt", KINDS)
@pytest.mark.parametrize("relu", [False, True])
def test_act8_codes_are_the_nearest_ties_to_even(relu, dt):
    """In whole numbers: 16-bit values and their block's largest often meet where a quotient lies
    exactly between two codes.  (Quotients that are not there but within 2^-15 of it may go as if.)"""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.randn(4000, 512, generator=g, device="cuda") * torch.exp(torch.randn(4000, 1, generator=g, device="cuda"))).to(dt)
    x[:64] = (torch.randint(-255, 256, (64, 512), generator=g, device="cuda") / 2).to(dt)  # halves: many ties
    x[:64, ::64] = 255.0 if relu else 127.0
    q = sf.quantize_act8(x, relu=relu)
    codes = (q.codes if relu else q.codes.view(torch.int8)).long().view(-1, 64)
    top = 255 if relu else 127
    v = (x.float() * 2.0 ** 20).round().long().view(-1, 64)  # exact, but for bits below 2^-20 of values that small
    x20 = v.double() * 2.0 ** -20
    exact = (x20 == x.double().view(-1, 64)).all(1)  # blocks without such
    if relu:
        v = v.clamp_min(0)
    m = v.abs().amax(1, keepdim=True)
    exact &= m[:, 0] > 0
    two = 2 * top * v.abs()  # twice the quotient, times m
    k = two // (2 * m).clamp_min(1)
    rest = two - 2 * m * k   # 0 .. 2 m: the half is m
    want = torch.where(rest > m, k + 1, torch.where(rest < m, k, k + (k & 1)))
    if relu:
        want = torch.where((v > 0) & (want < 1), 1, want)
    near_half = (rest != m) & ((rest - m).abs().double() < 2 * m.double() * 2.0 ** -15)
    ok = (codes == want * v.sign()) | (near_half & ((codes.abs() - want).abs() <= 1))
    assert exact.sum() > 1000 and (rest[exact] == m[exact].expand_as(rest[exact])).sum() > 1000  # the ties are there
    assert ok[exact].all(), f"{int((~ok[exact]).sum())} codes of {int(exact.sum()) * 64}"


@pytest.mark.parametrize("T,n,spread", [(3, 72, 0.0), (130, 200, 1.0), (257, 520, 3.0), (40, 64, 8.0)])
def test_full_codes_hold_what_they_promise(T, n, spread):
    """relu(G) and U as they are kept, of any size: one product each, exact in 32 bits, under
    factors from 2^-60 to 2^60 a token and neurons spread over many octaves."""
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = torch.zeros(T, 8, device="cuda", dtype=torch.bfloat16)
    x[:, 0] = (r(T) * 2.0 ** torch.randint(-60, 61, (T,), generator=g, device="cuda")).bfloat16()
    wg, wu = (torch.zeros(n, 8, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for w in (wg, wu):
        w[:, 0] = (r(n) * torch.exp(spread * r(n))).clamp(-2.0 ** 60, 2.0 ** 60).bfloat16()
    x[0], wg[5], wu[7] = 0, 0, -0.0
    if T > 100:  # largest values that round up to a power of two
        x[1, 0], wg[64:128, 0], wu[64:128, 0] = 255 / 256, 1 + 127 / 128, -1 - 127 / 128
    _, s = sf.gated_ffn_forward(x, wg, wu, torch.zeros(8, n, device="cuda", dtype=torch.bfloat16), save="full")
    G, U = (x[:, :1].double() @ w[:, :1].double().t() for w in (wg, wu))
    for codes, scales, v, bits, signed in ((s.r, s.r_scales, G.clamp_min(0), 13, False), (s.u, s.u_scales, U, 12, True)):
        c = codes[:, :n].long() & 0xffff
        m = c & 0x7fff if signed else c
        meet = 10 << (bits - 1)
        word = torch.minimum(2 * m, m + meet) << (23 - bits)
        P = scales.double().repeat_interleave(64, 1)[:, :n]
        held = word.int().view(torch.float32).double() * 2.0 ** 115 * P
        if signed:
            held = torch.where(c >= 0x8000, -held, held)
        else:
            assert torch.equal(c > 0, v > 0)
        # the scale: the power of two at or below the largest (or the next, which that rounds to), 2^-101 at least
        top = torch.nn.functional.pad(v.abs(), (0, -n % 64)).view(T, -1, 64).amax(2)
        S = scales.double()
        assert torch.equal(torch.frexp(S).mantissa, torch.full_like(S, 0.5)) and (S >= 2.0 ** -101).all()
        assert ((S <= top * (1 + 2.0 ** -bits)) & (top < 2 * S) | (S == 2.0 ** -101) & (top < 2 * S)).all()
        step = torch.where(v.abs() >= P / 4, 2.0 ** -(bits + 1), 2.0 ** -bits).double()
        tol = torch.maximum(v.abs() * step, P * 2.0 ** -(bits + 11))
        if not signed:
            tol = torch.where(c == 1, torch.maximum(tol, P * 2.0 ** -(bits + 10)), tol)  # lifted: a whole step
        assert ((held - v).abs() <= tol * (1 + 2.0 ** -10)).all()
    assert sf.dense_error() == 0


def test_error_word_made_in_inference_mode_can_be_cleared(monkeypatch):
    from activation_sparse_ffn_threshold_b200 import dense
    monkeypatch.setattr(dense, "_err_words", {})
    monkeypatch.setattr(dense, "_err_ptrs", {})
    x, wg, wu, wd, b, dy = layer(4, 64, 128, torch.float16, seed=1)
    with torch.inference_mode():  # the first call, which allocates the word
        sf.gated_ffn_forward(x, wg, wu, wd, b)
        torch.cuda.synchronize()
        dense._err_words[torch.cuda.current_device()].fill_(5)  # as a wait that ran out would
    assert sf.dense_error() == 5 and sf.dense_error() == 0
