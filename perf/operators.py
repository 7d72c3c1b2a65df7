"""The dense gated FFN, its training step with plain and with 8-bit saved activations, the 8-bit
activation blocks by themselves, and the microscaled 4-bit linear layer: cases, plain forms, exact values.

``own = False`` computes an operator in plain torch operations in 32 bits, rounded once at the
end; ``own = True`` calls the framework.

    gated FFN   G = X Wg^T + b, U = X Wu^T, H = relu(G) * U, Y = H Wd^T
    its step    dH = dY Wd, dU = dH * relu(G), dG = dH * U * [G > 0], dX = dG Wg + dU Wu,
                dWg = dG^T X, dWu = dU^T X, dWd = dY^T H, db = sum over tokens of dG
    act8        64 values share a scale: max|v| / 127 with signed codes, or for relu(v)
                max / 255 with codes 0..255, where a positive value keeps a code of at least 1
    mxfp4       32 values share a power of two 2^(floor(log2 max|v|) - 2); each is held as one of
                0, .5, 1, 1.5, 2, 3, 4, 6 with a sign, rounded to nearest, ties to the even code
"""
import math

import torch

own = False

KINDS = {"f16": torch.float16, "bf16": torch.bfloat16}
BLOCK8 = 64
BLOCK4 = 32


def listed():
    return [
        # one token through all neurons of a 7B-shaped layer: decode without a predictor, bound by the weights' bytes
        {"name": "ffn_1_token", "op": "ffn", "T": 1, "d": 4096, "n": 11008, "dtype": "f16", "pad": 0},
        # a decode batch on a 70B-shaped layer: still bound by the weights, odd token count
        {"name": "ffn_37_tokens", "op": "ffn", "T": 37, "d": 8192, "n": 28672, "dtype": "bf16", "pad": 0},
        # a prompt whose length fills no tile, rows of a wider buffer
        {"name": "ffn_prompt_2000", "op": "ffn", "T": 2000, "d": 4096, "n": 11008, "dtype": "f16", "pad": 64},
        # fine-tuning a small layer on a short ragged sequence: launches and latency count
        {"name": "step_257_small", "op": "step", "T": 257, "d": 512, "n": 2048, "dtype": "f16", "pad": 0},
        # a training step of a 7B-shaped layer: bound by the tensor cores
        {"name": "step_4096", "op": "step", "T": 4096, "d": 4096, "n": 11008, "dtype": "bf16", "pad": 0},
        # the same two with the activations held in 8 bits between forward and backward
        {"name": "step8_1000_odd", "op": "step8", "T": 1000, "d": 1024, "n": 5000, "dtype": "f16", "pad": 0},
        {"name": "step8_4096", "op": "step8", "T": 4096, "d": 4096, "n": 11008, "dtype": "bf16", "pad": 0},
        # one short sequence's activations saved and restored (latency), last block of a row short
        {"name": "act8_small_odd", "op": "act8", "T": 301, "d": 1000, "relu": False, "dtype": "f16"},
        # a whole layer's hidden activations saved and restored: bound by bytes
        {"name": "act8_hidden", "op": "act8", "T": 8192, "d": 11008, "relu": True, "dtype": "bf16"},
        # 4-bit weights: one token (bytes), a decode batch with an odd output width, a prompt (tensor cores)
        {"name": "mxfp4_1_token", "op": "mxfp4", "T": 1, "K": 4096, "N": 11008, "dtype": "f16"},
        {"name": "mxfp4_77_odd", "op": "mxfp4", "T": 77, "K": 4096, "N": 4099, "dtype": "bf16"},
        {"name": "mxfp4_prompt", "op": "mxfp4", "T": 4096, "K": 8192, "N": 28672, "dtype": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    """Another case of the listed ones' ranges; widths in steps of 8 (of 32 for mxfp4's K)."""
    op = rng.choice(["ffn", "step", "step8", "act8", "mxfp4"])
    kind = rng.choice(["f16", "bf16"])
    while True:
        if op == "act8":
            case = {"op": op, "T": _log(rng, 1, 8192), "d": _log(rng, 8, 28672), "relu": rng.random() < 0.5,
                    "dtype": kind}
            if case["T"] * case["d"] <= 8192 * 11008:
                return case
        elif op == "mxfp4":
            case = {"op": op, "T": _log(rng, 1, 4096), "K": _log(rng, 64, 8192, 32), "N": _log(rng, 64, 28672),
                    "dtype": kind}
            return case
        else:
            case = {"op": op, "T": _log(rng, 1, 4096), "d": _log(rng, 64, 8192, 8), "n": _log(rng, 64, 28672, 8),
                    "dtype": kind, "pad": rng.choice([0, 0, 8, 64])}
            if case["T"] * case["d"] * case["n"] <= 4096 * 4096 * 11008:
                return case


# ------------------------------------------------------------------------------------------ inputs
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _mx_inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    K, N = case["K"], case["N"]
    x = _normal(g, case["T"], K)
    x[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device="cuda")] *= 8.0  # outlier channels
    return x.to(KINDS[case["dtype"]]), (_normal(g, N, K) / math.sqrt(K)).to(KINDS[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = KINDS[case["dtype"]]
    T, s = case["T"], {"case": case}
    if case["op"] == "act8":
        x = _normal(g, T, case["d"]) * torch.exp(0.5 * _normal(g, 1, case["d"]))
        s["x"] = x.to(dt)
        return s
    if case["op"] == "mxfp4":
        s["x"], w = _mx_inputs(case, seed)
        if own:
            from activation_sparse_ffn_threshold_b200 import quantize_mxfp4
            s["w"] = quantize_mxfp4(w)
        else:
            s["w"] = _mx_codes(w.float())
        return s
    d, n = case["d"], case["n"]
    # The gate's operands lie on grids (x in sixteenths, gate weights and biases in powers of two near a
    # quarter of their deviation), so that its sums are exact in 32 bits in every order and a neuron at the
    # ReLU's border falls on the same side everywhere.  About 15% of the neurons are active.
    x = torch.zeros(T, d + case["pad"], device="cuda")
    x[:, :d] = (_normal(g, T, d) * 16).round().clamp(-64, 64) / 16
    s["x"] = x.to(dt)[:, :d]
    unit = 2.0 ** round(math.log2(0.25 / math.sqrt(d)))
    s["w_gate"] = ((_normal(g, n, d) / math.sqrt(d) / unit).round().clamp(-24, 24) * unit).to(dt)
    s["w_up"] = (_normal(g, n, d) / math.sqrt(d)).to(dt)
    s["w_down"] = (_normal(g, d, n) / math.sqrt(n)).to(dt)
    s["b"] = (((_normal(g, n) * 0.3 - 1.04) * 32).round() / 32).to(dt)
    if case["op"] != "ffn":
        s["dy"] = (_normal(g, T, d) * 0.1).to(dt)
    return s


# ------------------------------------------------------------------------------------- plain forms
def _act8_plain(v, relu):
    """The values that act8 holds for v [T, C] (32 bits in and out)."""
    T, C = v.shape
    pad = -C % BLOCK8
    v = torch.nn.functional.pad(v, (0, pad)).view(T, -1, BLOCK8)
    if relu:
        v = v.clamp_min(0.0)
        s = v.amax(2, keepdim=True) / 255.0
        c = torch.round(v / torch.where(s > 0, s, 1.0)).clamp(0, 255)
        c = torch.where((v > 0) & (c < 1), 1.0, c)
    else:
        s = v.abs().amax(2, keepdim=True) / 127.0
        c = torch.round(v / torch.where(s > 0, s, 1.0)).clamp(-127, 127)
    return (c * s).view(T, -1)[:, :C]


def _mx_scale(e):
    """2^e in 32 bits for whole e in [-127, 127], from its bits (2^-127 is a subnormal)."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _mx_codes(v):
    """(exponents [R, K/32], codes [R, K/2], two 4-bit codes a byte) of v [R, K] in 32 bits."""
    R, K = v.shape
    v = v.view(R, K // BLOCK4, BLOCK4)
    top = v.abs().amax(2, keepdim=True)
    e = ((top.view(torch.int32) >> 23) - 129).clamp(-127, 127)  # the biased exponent, less 127 and 2
    a = v.abs() / _mx_scale(e)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    up = torch.bucketize(a, edges, right=True)   # an edge belongs to the upper code
    low = torch.bucketize(a, edges, right=False)  # an edge belongs to the lower code
    code = torch.where(up % 2 == 0, up, low)     # a tie goes to the even one
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).view(R, K)
    return e.view(R, -1), code[:, 0::2] | (code[:, 1::2] << 4)


def _mx_values(e, packed):
    steps = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=e.device)
    steps = torch.cat([steps, -steps])
    code = torch.stack([packed & 15, packed >> 4], 2).long()
    v = steps[code.view(e.shape[0], e.shape[1], BLOCK4)]
    return (v * _mx_scale(e).unsqueeze(2)).view(e.shape[0], -1)


def _ffn_plain(s):
    x, b = s["x"].float(), s["b"].float()
    wg, wu, wd = s["w_gate"].float(), s["w_up"].float(), s["w_down"].float()
    gate = x @ wg.t() + b
    up = x @ wu.t()
    return x, wg, wu, wd, gate, up, (gate.clamp_min(0.0) * up) @ wd.t()


def _step_plain(s, eight):
    dt = s["x"].dtype
    x, wg, wu, wd, gate, up, y = _ffn_plain(s)
    r = gate.clamp_min(0.0)
    if eight:
        x, r, up = _act8_plain(x, False), _act8_plain(gate, True), _act8_plain(up, False)
    dy = s["dy"].float()
    dh = dy @ wd
    du = dh * r
    dg = dh * up * (gate > 0)
    dx = dg @ wg + du @ wu
    out = (y, dx, dg.t() @ x, du.t() @ x, dy.t() @ (r * up), dg.sum(0))
    return tuple(o.to(dt) for o in out)


def _run_plain(s):
    op, x = s["case"]["op"], s["x"]
    if op == "ffn":
        return _ffn_plain(s)[-1].to(x.dtype)
    if op == "act8":
        return _act8_plain(x.float(), s["case"]["relu"]).to(x.dtype)
    if op == "mxfp4":
        return (_mx_values(*_mx_codes(x.float())) @ _mx_values(*s["w"]).t()).to(x.dtype)
    return _step_plain(s, op == "step8")


def run(s):
    if not own:
        return _run_plain(s)
    import activation_sparse_ffn_threshold_b200 as sf
    case, x = s["case"], s["x"]
    op = case["op"]
    if op == "ffn":
        return sf.gated_ffn_forward(x, s["w_gate"], s["w_up"], s["w_down"], s["b"])[0]
    if op == "act8":
        return sf.dequantize_act8(sf.quantize_act8(x, relu=case["relu"]))
    if op == "mxfp4":
        return sf.mxfp4_linear(x, s["w"])
    y, saved = sf.gated_ffn_forward(x, s["w_gate"], s["w_up"], s["w_down"], s["b"],
                                    save="act8" if op == "step8" else "full")
    return (y,) + tuple(sf.gated_ffn_backward(s["dy"], saved, s["w_gate"], s["w_up"], s["w_down"]))


def work(case):
    T = case["T"]
    if case["op"] == "act8":
        v = T * case["d"]
        return {"bytes": 4 * v + 2 * (v + v / 16), "flops": 4 * v}  # 16-bit in and out, codes and scales there and back
    if case["op"] == "mxfp4":
        K, N = case["K"], case["N"]
        return {"bytes": 2 * T * K + N * K / 2 + N * K / 32 + 2 * T * N, "flops": 2 * T * N * K}
    d, n = case["d"], case["n"]
    if case["op"] == "ffn":
        return {"bytes": 2 * (3 * n * d + n + 2 * T * d), "flops": 6 * T * n * d}
    return {"bytes": 2 * (6 * n * d + 2 * n + 4 * T * d), "flops": 18 * T * n * d}


# ---------------------------------------------------------------------------------- exact values
def _blocks64(v, relu):
    """act8's values from its definition, block by block of 64 columns, in 64 bits."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], BLOCK8):
        p = v[:, c:c + BLOCK8]
        p = torch.relu(p) if relu else p
        step = p.abs().max(dim=1).values[:, None] / (255 if relu else 127)
        k = torch.nan_to_num(p / step, nan=0.0).round()
        if relu:
            k = torch.maximum(k, (p > 0).double())
        out[:, c:c + BLOCK8] = k * step
    return out


def _micro64(v):
    """mxfp4's values from its definition in 64 bits: each magnitude rounded on its binade's grid."""
    R, K = v.shape
    p = v.reshape(-1, BLOCK4)
    top = p.abs().max(dim=1).values
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, 0).clamp(-127, 127).long()
    scale = ((e + 1023) << 52).view(torch.float64)[:, None]  # 2^e exactly
    a = p.abs() / scale
    grid = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    q = torch.minimum((a / grid).round() * grid, torch.tensor(6.0, dtype=torch.float64, device=v.device))
    return (q * torch.sign(p) * scale).reshape(R, K)


def exact(case, seed):
    if case["op"] == "mxfp4":  # from the weights themselves: a state keeps only what they were quantised to
        x, w = _mx_inputs(case, seed)
        return _micro64(x.double()) @ _micro64(w.double()).t()
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "act8":
        return _blocks64(x, case["relu"])
    wg, wu, wd, b = (s[k].double() for k in ("w_gate", "w_up", "w_down", "b"))
    pre, up = torch.addmm(b, x, wg.t()), torch.mm(x, wu.t())
    on = (pre > 0).double()
    y = torch.mm(pre * on * up, wd.t())
    if case["op"] == "ffn":
        return y
    dy = s["dy"].double()
    r = pre * on
    if case["op"] == "step8":
        x, r, up = _blocks64(x, False), _blocks64(pre, True), _blocks64(up, False)
    dh = torch.mm(dy, wd)
    du, dg = dh * r, dh * up * on
    return (y, torch.addmm(torch.mm(dg, wg), du, wu), torch.mm(dg.t(), x), torch.mm(du.t(), x),
            torch.mm(dy.t(), r * up), dg.sum(dim=0))
