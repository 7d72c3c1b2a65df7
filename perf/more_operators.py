"""The linear layer with its epilogue, the norms around a block and the clipping of gradients: cases,
plain forms, exact values.

``own = False`` computes an operator in plain torch operations in 32 bits, rounded once at the
end; ``own = True`` calls the framework.

    linear    Z = X W^T + b, Y = act(Z) + residual; act: none, relu, gelu (z Phi(z)), silu (z / (1 + e^-z))
    its step  dZ = dY act'(Z), dX = dZ W, dW = dZ^T X, db = sum over tokens of dZ
    norm      R = a X + c gate * post(Z), H = pre(R); post and pre: none, "rms" (v / sqrt(mean v^2 + eps) * w + b)
              or "layer" ((v - mean) / sqrt(var + eps) * w + b)
    its step  the gradients of X, Z, the gate, and both norms' weights and biases from those of R and H
    clip      n = scale sqrt(sum over all tensors of g^2), out = g scale min(1, max_norm / (n + 1e-6))
"""
import math

import torch

own = False

KINDS = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def listed():
    return [
        # one token through the first product of an OPT-6.7B-shaped layer: bound by the weights' bytes
        {"name": "linear_1_token", "op": "linear", "T": 1, "K": 4096, "N": 16384, "act": "relu", "bias": True,
         "res": "none", "dtype": "f16", "pad": 0},
        # a decode batch through the second product of an OPT-30B-shaped layer, onto an fp32 residual stream
        {"name": "linear_50_tokens_onto_f32", "op": "linear", "T": 50, "K": 28672, "N": 7168, "act": "none",
         "bias": True, "res": "f32", "dtype": "f16", "pad": 0},
        # a prompt whose length fills no tile, from rows of a wider buffer, with a smooth activation
        {"name": "linear_prompt_1999", "op": "linear", "T": 1999, "K": 4096, "N": 16384, "act": "gelu", "bias": True,
         "res": "none", "dtype": "bf16", "pad": 64},
        # fine-tuning a small layer on a short sequence, odd output width: launches and latency count
        {"name": "linear_step_small_odd", "op": "linear_step", "T": 333, "K": 512, "N": 2047, "act": "silu",
         "bias": True, "res": "same", "dtype": "f16", "pad": 0},
        # a training step of an OPT-6.7B-shaped layer's first product: bound by the tensor cores
        {"name": "linear_step_4096", "op": "linear_step", "T": 4096, "K": 4096, "N": 16384, "act": "relu",
         "bias": True, "res": "none", "dtype": "bf16", "pad": 0},
        # decode: the sparse FFN's fp32 output joins the fp32 residual, the next layer's input is normed (latency)
        {"name": "norm_1_token", "op": "norm", "T": 1, "d": 4096, "pre": "rms", "post": "none", "gate": "none",
         "bias": False, "z": True, "x32": True, "z32": True, "a": 1.0, "c": 1.0, "dtype": "f16"},
        # a prompt through a 70B-shaped block's end: norms on both sides, a gate per channel
        {"name": "norm_prompt_4000", "op": "norm", "T": 4000, "d": 8192, "pre": "rms", "post": "rms", "gate": "vec",
         "bias": False, "z": True, "x32": False, "z32": False, "a": 1.0, "c": 0.5, "dtype": "bf16"},
        # a short sequence's step with LayerNorm and biases, a width that no vector load divides
        {"name": "norm_step_small_odd", "op": "norm_step", "T": 301, "d": 1001, "pre": "layer", "post": "none",
         "gate": "none", "bias": True, "z": True, "x32": True, "z32": False, "a": 1.0, "c": 1.0, "dtype": "f16"},
        # a training step's block end at a 7B width: bound by bytes
        {"name": "norm_step_8192", "op": "norm_step", "T": 8192, "d": 4096, "pre": "rms", "post": "rms",
         "gate": "vec", "bias": False, "z": True, "x32": False, "z32": False, "a": 1.0, "c": 1.0, "dtype": "bf16"},
        # the gradients of a small stack: many tensors, odd sizes, latency
        {"name": "clip_small_stack", "op": "clip", "layers": 8, "d": 509, "n": 2039, "kind": "f16", "scale": 1 / 1024,
         "max_norm": 1.0},
        # one 7B-shaped ReGLU layer's gradients (norms and biases in fp32), not clipped
        {"name": "clip_layer", "op": "clip", "layers": 1, "d": 4096, "n": 11008, "kind": "bf16", "scale": 1.0,
         "max_norm": 1e6},
        # four such layers, clipped: bound by bytes
        {"name": "clip_stack", "op": "clip", "layers": 4, "d": 4096, "n": 11008, "kind": "bf16", "scale": 1.0,
         "max_norm": 1.0},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(hi, max(lo, round(v / step) * step)))


def draw(rng):
    """Another case of the listed ones' ranges; K in steps of 8."""
    op = rng.choice(["linear", "linear_step", "norm", "norm_step", "clip"])
    dtype = rng.choice(["f16", "bf16"])
    while True:
        if op in ("linear", "linear_step"):
            case = {"op": op, "T": _log(rng, 1, 4096), "K": _log(rng, 64, 28672, 8), "N": _log(rng, 64, 28672),
                    "act": rng.choice(["none", "relu", "gelu", "silu"]), "bias": rng.random() < 0.7,
                    "res": rng.choice(["none", "same", "f32"]), "dtype": dtype, "pad": rng.choice([0, 0, 8, 64])}
            if case["T"] * case["K"] * case["N"] <= 4096 * 4096 * 16384:
                return case
        elif op == "clip":
            case = {"op": op, "layers": rng.randint(1, 8), "d": _log(rng, 8, 8192), "n": _log(rng, 8, 28672),
                    "kind": rng.choice(["f16", "bf16", "f32"]), "scale": rng.choice([1.0, 0.25]),
                    "max_norm": rng.choice([0.5, 1.0, 1e6])}
            if case["layers"] * case["d"] * case["n"] * (2 if case["kind"] == "f32" else 1) <= 4 * 4096 * 11008:
                return case
        else:
            z = rng.random() < 0.85
            case = {"op": op, "T": _log(rng, 1, 8192), "d": _log(rng, 8, 8192),
                    "pre": rng.choice(["rms", "layer"] + ["none"] * z), "post": rng.choice(["none", "rms", "layer"]),
                    "gate": rng.choice(["none", "vec", "token"]), "bias": rng.random() < 0.5, "z": z,
                    "x32": rng.random() < 0.5, "z32": rng.random() < 0.25, "a": rng.choice([1.0, 1.0, 0.75]),
                    "c": rng.choice([1.0, 1.0, 0.5]), "dtype": dtype}
            if not z:
                case.update(post="none", gate="none", a=1.0, c=1.0)
            if case["T"] * case["d"] <= (8192 * 4096 if op == "norm_step" else 4000 * 8192):
                return case


# ------------------------------------------------------------------------------------------ inputs
def _shapes(case):
    """The gradients of a stack of gated layers with a norm each: (shape, held in 32 bits)."""
    d, n, wide = case["d"], case["n"], case["kind"] == "f32"
    return [((n, d), wide), ((n, d), wide), ((d, n), wide), ((n,), True), ((d,), True)] * case["layers"]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": case}
    if case["op"] == "clip":
        dt = KINDS.get(case["kind"], torch.float32)
        size = 4.0 / case["scale"] / math.sqrt(sum(math.prod(shape) for shape, _ in _shapes(case)))
        s["grads"] = [(normal(*shape) * size * math.exp(0.5 * math.sin(i))).to(torch.float32 if wide else dt)
                      for i, (shape, wide) in enumerate(_shapes(case))]
        s["out"] = [torch.empty_like(t) for t in s["grads"]]
        return s
    dt, T = KINDS[case["dtype"]], case["T"]
    if case["op"] in ("linear", "linear_step"):
        K, N = case["K"], case["N"]
        # For a ReLU the operands lie on grids (x in sixteenths, weights in powers of two near a quarter of
        # their deviation), so that the sums are exact in 32 bits in every order and a value at the ReLU's
        # border falls on the same side everywhere.
        on_grid = case["act"] == "relu"
        x = torch.zeros(T, K + case["pad"], device="cuda")
        x[:, :K] = (normal(T, K) * 16).round().clamp(-64, 64) / 16 if on_grid else normal(T, K)
        s["x"] = x.to(dt)[:, :K]
        w = normal(N, K) / math.sqrt(K)
        if on_grid:
            unit = 2.0 ** round(math.log2(0.25 / math.sqrt(K)))
            w = (w / unit).round().clamp(-24, 24) * unit
        s["w"] = w.to(dt)
        s["b"] = (((normal(N) * 0.3 - 0.5) * 32).round() / 32).to(dt) if case["bias"] else None
        s["res"] = None if case["res"] == "none" else normal(T, N).to(torch.float32 if case["res"] == "f32" else dt)
        if case["op"] == "linear_step":
            s["dy"] = (normal(T, N) * 0.1).to(torch.float32 if case["res"] == "f32" else dt)
        return s
    d = case["d"]
    loud = 1.0 + 20.0 * (torch.rand(d, generator=g, device="cuda") < 2.0 / d)  # a few outlier channels
    xt, zt = torch.float32 if case["x32"] else dt, torch.float32 if case["z32"] else dt
    s["x"] = (normal(T, d) * loud + 0.2 * normal(d)).to(xt)
    s["z"] = (normal(T, d) * torch.exp(0.5 * normal(T, 1)) + 0.1).to(zt) if case["z"] else None
    s["gate"] = {"none": lambda: None, "vec": lambda: (1 + 0.2 * normal(d)).to(dt),
                 "token": lambda: torch.sigmoid(normal(T, d)).to(dt)}[case["gate"]]()
    for k, kind in (("", case["pre"]), ("post_", case["post"])):
        s[k + "w"] = (1 + 0.1 * normal(d)).to(dt) if kind != "none" else None
        s[k + "b"] = (0.1 * normal(d)).to(dt) if kind != "none" and case["bias"] else None
    if case["op"] == "norm_step":
        s["dr"] = (normal(T, d) * 0.1).to(xt)
        s["dh"] = (normal(T, d) * 0.1).to(dt) if case["pre"] != "none" else None
    return s


# ------------------------------------------------------------------------------------- plain forms
def _phi(z):
    return 0.5 * torch.erfc(z * -math.sqrt(0.5))


def _act(z, act):
    """(act(z), act'(z))."""
    if act == "relu":
        return z.clamp_min(0.0), (z > 0).float()
    if act == "gelu":
        p = _phi(z)
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    return z, torch.ones_like(z)


def _linear_plain(s):
    case, x, w, b, res = s["case"], s["x"], s["w"], s["b"], s["res"]
    z = x.float() @ w.float().t()
    if b is not None:
        z = z + b.float()
    y, slope = _act(z, case["act"])
    if res is not None:
        y = y + res.float()
    y = y.to(x.dtype if res is None else res.dtype)
    if case["op"] == "linear":
        return y
    dz = s["dy"].float() * slope
    return (y, (dz @ w.float()).to(x.dtype), (dz.t() @ x.float()).to(w.dtype),
            dz.sum(0).to(b.dtype) if b is not None else None)


def _normed(v, kind):
    """(the normed rows, what they were divided by)."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    s = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * s, s


def _norm_back(u, hat, s, kind):
    """The gradient of a normed row's input from that of the normed row."""
    d = u - hat * (u * hat).mean(1, keepdim=True)
    if kind == "layer":
        d = d - u.mean(1, keepdim=True)
    return s * d


def _norm_plain(s):
    case = s["case"]
    dt = KINDS[case["dtype"]]
    f = {k: v.float() for k, v in s.items() if isinstance(v, torch.Tensor)}
    r, p = f["x"], None
    if "z" in f:
        p = f["z"]
        if case["post"] != "none":
            zhat, zs = _normed(p, case["post"])
            p = zhat * f["post_w"] + f.get("post_b", 0.0)
        r = case["a"] * r + case["c"] * (p * f["gate"] if "gate" in f else p)
    h = None
    if case["pre"] != "none":
        hat, hs = _normed(r, case["pre"])
        h = hat * f["w"] + f.get("b", 0.0)
    R = s["x"] if p is None else r.to(s["x"].dtype)
    if case["op"] == "norm":
        return R, None if h is None else h.to(dt)
    D = f["dr"]
    dw = db = dz = dgate = dpw = dpb = None
    if h is not None:
        dw, db = (f["dh"] * hat).sum(0).to(dt), f["dh"].sum(0).to(dt) if "b" in f else None
        D = D + _norm_back(f["dh"] * f["w"], hat, hs, case["pre"])
    if p is not None:
        dp = case["c"] * D
        if "gate" in f:
            dgate = dp * p
            dgate = (dgate if case["gate"] == "token" else dgate.sum(0)).to(dt)
            dp = dp * f["gate"]
        if case["post"] != "none":
            dpw, dpb = (dp * zhat).sum(0).to(dt), dp.sum(0).to(dt) if "post_b" in f else None
            dp = _norm_back(dp * f["post_w"], zhat, zs, case["post"])
        dz = dp.to(s["z"].dtype)
    dx = (case["a"] * D if p is not None else D).to(s["x"].dtype)
    return R, None if h is None else h.to(dt), dx, dz, dgate, dw, db, dpw, dpb


def _clip_plain(s):
    case = s["case"]
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    n = (case["scale"] * total.sqrt()).float()
    k = case["scale"] * (case["max_norm"] / (n + 1e-6)).clamp(max=1.0)
    return [n] + [(g.float() * k).to(g.dtype) for g in s["grads"]]


def _run_plain(s):
    op = s["case"]["op"]
    return _clip_plain(s) if op == "clip" else _norm_plain(s) if op in ("norm", "norm_step") else _linear_plain(s)


def run(s):
    if not own:
        return _run_plain(s)
    import activation_sparse_ffn_threshold_b200 as sf
    case = s["case"]
    op = case["op"]
    if op == "clip":
        return [sf.clip_grad_norm(s["grads"], case["max_norm"], scale=case["scale"], out=s["out"])] + s["out"]
    if op == "linear":
        return sf.linear_forward(s["x"], s["w"], s["b"], act=case["act"], residual=s["res"])[0]
    if op == "linear_step":
        y, saved = sf.linear_forward(s["x"], s["w"], s["b"], act=case["act"], residual=s["res"], save=True)
        return (y,) + tuple(sf.linear_backward(s["dy"], saved, s["w"]))
    r, h, saved = sf.residual_norm_forward(
        s["x"], s["z"], pre=case["pre"], w=s["w"], b=s["b"], post=case["post"], post_w=s["post_w"],
        post_b=s["post_b"], gate=s["gate"], residual_scale=case["a"], branch_scale=case["c"], eps=EPS,
        save=op == "norm_step")
    if op == "norm":
        return r, h
    return (r, h) + tuple(sf.residual_norm_backward(s["dr"], s["dh"], saved))


def work(case):
    if case["op"] == "clip":
        sizes = [(math.prod(shape), 4 if wide else 2) for shape, wide in _shapes(case)]
        return {"bytes": sum(2 * n * e for n, e in sizes) + 4, "flops": sum(3 * n for n, _ in sizes)}
    T, step = case["T"], case["op"].endswith("step")
    if case["op"] in ("linear", "linear_step"):
        K, N = case["K"], case["N"]
        ye = 4 if case["res"] == "f32" else 2
        res = 0 if case["res"] == "none" else ye * T * N
        v = 2 * T * K + 2 * N * K + ye * T * N + res + 2 * N * case["bias"]
        if step:
            v += ye * T * N + 2 * T * K + 2 * N * K + 2 * N * case["bias"]
        return {"bytes": v, "flops": (6 if step else 2) * T * K * N}
    d, z = case["d"], case["z"]
    xe, ze = 4 if case["x32"] else 2, 4 if case["z32"] else 2
    pre, token = case["pre"] != "none", case["gate"] == "token"
    norms = (pre + (case["post"] != "none")) * (1 + case["bias"]) + (case["gate"] == "vec")
    v = T * d * (xe + (ze + xe if z else 0) + 2 * pre + 2 * token) + 2 * d * norms
    if step:
        v += T * d * (2 * xe + ze * z + 2 * pre + 2 * token) + 2 * d * norms
    return {"bytes": v, "flops": (40 if step else 15) * T * d}


# ---------------------------------------------------------------------------------- exact values
def _slope64(z, act):
    """act(z) and its derivative in 64 bits, by autograd of the definition."""
    with torch.enable_grad():
        v = z.detach().requires_grad_()
        y = {"none": lambda: v * 1.0, "relu": lambda: torch.relu(v), "silu": lambda: v * torch.sigmoid(v),
             "gelu": lambda: v * 0.5 * (1.0 + torch.erf(v / math.sqrt(2.0)))}[act]()
        (d,) = torch.autograd.grad(y.sum(), v)
    return y.detach(), d


def _linear64(case, s):
    x, w = s["x"].double(), s["w"].double()
    z = torch.mm(x, w.t())
    if s["b"] is not None:
        z += s["b"].double()
    y, slope = _slope64(z, case["act"])
    del z
    if s["res"] is not None:
        y = y + s["res"].double()
    if case["op"] == "linear":
        return y
    dz = s["dy"].double().mul_(slope)
    return (y, torch.mm(dz, w), torch.mm(dz.t(), x), None if s["b"] is None else dz.sum(dim=0))


def _norm64(case, s):
    """R, H and, for a step, their gradients by autograd of the definition."""
    leaves = {k: s[k].double().requires_grad_() for k in ("x", "z", "gate", "w", "b", "post_w", "post_b")
              if s[k] is not None}

    def norm(v, kind, w, b):
        m = v.mean(dim=1)[:, None] if kind == "layer" else 0.0
        q = ((v - m) / torch.sqrt(((v - m) ** 2).sum(dim=1) / v.shape[1] + EPS)[:, None]) * leaves[w]
        return q + leaves[b] if b in leaves else q

    step = case["op"] == "norm_step"
    with torch.set_grad_enabled(step):
        r = leaves["x"]
        if "z" in leaves:
            p = leaves["z"] if case["post"] == "none" else norm(leaves["z"], case["post"], "post_w", "post_b")
            r = case["a"] * r + case["c"] * (p * leaves["gate"] if "gate" in leaves else p)
        h = None if case["pre"] == "none" else norm(r, case["pre"], "w", "b")
        if not step:
            return r.detach(), None if h is None else h.detach()
        loss = (r * s["dr"].double()).sum()
        if h is not None:
            loss = loss + (h * s["dh"].double()).sum()
        grads = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    return (r.detach(), None if h is None else h.detach()) + tuple(
        grads.get(k) for k in ("x", "z", "gate", "w", "b", "post_w", "post_b"))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        n = case["scale"] * math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s["grads"]))
        k = min(1.0, case["max_norm"] / (n + 1e-6))
        return [n] + [g.double().mul_(case["scale"] * k) for g in s["grads"]]
    return (_norm64 if case["op"] in ("norm", "norm_step") else _linear64)(case, s)
