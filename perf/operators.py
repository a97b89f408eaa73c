"""The block norm, block join, orthogonalisation and Muon update cases that are timed and checked.

Layout is the library's: activations [N, C, H, W] whose C channels are `groups` equal blocks, weights
[C_out, C_in/groups, kH, kW], which the optimiser reads as `groups` matrices of C_out/groups rows and
C_in/groups * kH * kW columns.

  norm   y = x * r * weight,  r = 1 / sqrt(mean over the group's channels of x^2 + eps), at each position.
         Its gradient adds the one that reaches x along the residual branch.
  join   the end of a residual block and the norm that opens the next one:
         out = res + scale * act(gate) * (h * r(h) * weight),  next = out * r(out) * next_weight
  orth   steps of X <- a X + (b A + c A A) X, A = X X^T, from X = g / (|g| + eps), on the shorter side
  muon   m' = beta m + g,  u = g + beta m',  w' = w (1 - lr decay) - lr scale orth(u)
"""
import math

import torch

own = False

EPS = 1e-6
NS_EPS = 1e-7
NS = (3.4445, -4.7750, 2.0315)
STEPS = 5
LR, BETA, DECAY = 5e-4, 0.95, 0.1


def _act(name, op, dtype, n, c, h, w, groups, gate="none", act="none"):
    case = {"op": op, "dtype": dtype, "n": n, "c": c, "h": h, "w": w, "groups": groups, "gate": gate, "act": act}
    return dict(case, name=name) if name else case


def _mat(name, op, dtype, co, ci, kh, kw, groups):
    case = {"op": op, "dtype": dtype, "co": co, "ci": ci, "kh": kh, "kw": kw, "groups": groups}
    return dict(case, name=name) if name else case


def listed():
    return [
        # eight sequences, one new position each: latency
        _act("norm_token", "norm_fwd", "bf16", 8, 1024, 1, 1, 1),
        # the small fp32 layer with five groups of 20 channels
        _act("norm_tiny_g5", "norm_fwd", "f32", 2, 100, 28, 28, 5),
        # the input of the 2-group 5x5 layer, a plane of 729 positions: rows never aligned
        _act("norm_bwd_27x27_g2", "norm_bwd", "bf16", 128, 96, 27, 27, 2),
        # a large bottleneck stage, gated: forward and backward
        _act("join_56x56", "join_fwd", "bf16", 64, 256, 56, 56, 1, "full", "silu"),
        _act("join_bwd_56x56", "join_bwd", "bf16", 64, 256, 56, 56, 1, "full", "silu"),
        # a late stage in fp32 with one gate a channel and image
        _act("join_bwd_7x7_f32", "join_bwd", "f32", 32, 1024, 7, 7, 1, "channel", "sigmoid"),
        # 32 groups of 4 x 36: the smallest matrices
        _mat("orth_resnext_g32", "orth", "f32", 128, 128, 3, 3, 32),
        # the 2-group 5x5 layer: 128 x 1200
        _mat("orth_alexnet_g2", "orth", "f32", 256, 96, 5, 5, 2),
        # the fully connected layer of 4096 x 9216
        _mat("orth_fc", "orth", "bf16", 4096, 256, 6, 6, 1),
        # the dense 3x3 layer: 64 x 576
        _mat("muon_dense3x3", "muon", "f32", 64, 64, 3, 3, 1),
        # a 1x1 expansion: taller than wide
        _mat("muon_1x1_64to256", "muon", "f32", 256, 64, 1, 1, 1),
        # a wide 3x3 layer: 1024 x 4608
        _mat("muon_3x3_512to1024", "muon", "f32", 1024, 512, 3, 3, 1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "join_fwd", "join_bwd", "orth", "muon"])
    if op in ("orth", "muon"):
        dtype = "f32" if op == "muon" else rng.choice(["f32", "bf16"])
        groups = rng.choice([1, 1, 1, 2, 4, 32])
        k = rng.choice([1, 1, 3, 3, 5])
        co = _log(rng, 4, 2048 // groups if groups < 32 else 32)
        ci = _log(rng, 4, max(8, 2048 // (groups * k) if groups < 32 else 32))
        return _mat(None, op, dtype, co * groups, ci * groups, k, k, groups)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    groups = rng.choice([1, 1, 1, 2, 5, 32])
    c = _log(rng, 16 if groups == 1 else 2, 1536 // groups) * groups
    h = rng.choice([1, 1, 7, 13, 14, 27, 28, 56])
    w = _log(rng, 1, 4096) if h == 1 else h
    n = _log(rng, 1, 128)
    most = 24_000_000 if dtype == "bf16" else 12_000_000
    n = max(1, min(n, most // (c * h * w)))
    gate, act = "none", "none"
    if op.startswith("join"):
        gate = rng.choice(["none", "full", "channel"])
        act = "none" if gate == "none" else rng.choice(["none", "sigmoid", "silu"])
    return _act(None, op, dtype, n, c, h, w, groups, gate, act)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _dtype(case)

    def normal(shape, sd=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, device=dev).normal_(mean, sd, generator=gen).to(dtype)

    s = dict(case)
    if case["op"] in ("orth", "muon"):
        shape = (case["co"], case["ci"] // case["groups"], case["kh"], case["kw"])
        # a gradient: rows of unlike size
        rows = torch.exp(normal((case["co"], 1, 1, 1), 0.3))
        s["g"] = (normal(shape, 1e-3) * rows).to(dt)
        if case["op"] == "orth":
            s["out"] = torch.empty(shape, device=dev, dtype=torch.bfloat16)
            return s
        fan = shape[1] * shape[2] * shape[3]
        s["w"] = normal(shape, fan ** -0.5)
        s["m"] = normal(shape, 3e-3) * rows
        s["w_out"], s["m_out"] = torch.empty_like(s["w"]), torch.empty_like(s["m"])
        s["w_bf16"] = torch.empty(shape, device=dev, dtype=torch.bfloat16)
        return s
    shape = (case["n"], case["c"], case["h"], case["w"])
    c = case["c"]
    new = lambda d=dt: torch.empty(shape, device=dev, dtype=d)  # noqa: E731
    # a residual stream has a few channels far larger than the rest
    loud = 1.0 + 8.0 * (torch.rand((1, c, 1, 1), device=dev, generator=gen) < 0.02).float()
    s["weight"] = normal((c,), 0.2, 1.0)
    if case["op"].startswith("norm"):
        s["x"] = (normal(shape, 2.0) * loud).to(dt)
        if case["op"] == "norm_fwd":
            s["y"] = new()
        else:
            s["dy"], s["dres"] = normal(shape, dtype=dt), normal(shape, dtype=dt)
            s["dx"], s["dweight"] = new(), torch.empty((c,), device=dev)
        return s
    s["next_weight"] = normal((c,), 0.2, 1.0)
    s["scale"] = normal((c,), 0.1, 0.3)
    s["h_"] = normal(shape, 0.7, dtype=dt)
    s["z"] = None
    if case["gate"] != "none":
        s["z"] = normal(shape if case["gate"] == "full" else shape[:2], 1.5, dtype=dt)
    s["res"] = (normal(shape, 2.0) * loud).to(dt)  # the backward pass reads it as the forward's `out`
    if case["op"] == "join_fwd":
        s["out"], s["next"] = new(), new()
        return s
    s["dout"], s["dnext"] = normal(shape, dtype=dt), normal(shape, dtype=dt)
    s["dres"], s["dh"] = new(), new()
    s["dz"] = None
    if case["gate"] == "full":
        s["dz"] = new()
    elif case["gate"] == "channel":
        s["dz"] = torch.empty(shape[:2], device=dev)
    for k in ("dweight", "dscale", "dnext_weight"):
        s[k] = torch.empty((c,), device=dev)
    return s


# ---- the plain forms ------------------------------------------------------------


def _grouped(t, s):
    return t.float().view(s["n"], s["groups"], s["c"] // s["groups"], -1)


def _channels(v, s):
    return v.view(1, s["groups"], s["c"] // s["groups"], 1)


def _rms(t):
    return torch.rsqrt((t * t).mean(2, keepdim=True) + EPS)


def _shape(s):
    return s["n"], s["c"], s["h"], s["w"]


def _norm_fwd(s):
    x = _grouped(s["x"], s)
    return {"y": (x * _rms(x) * _channels(s["weight"], s)).view(_shape(s)).to(s["x"].dtype)}


def _norm_grad(x, weight, dy):
    """(dx, dweight) of y = x r weight, all in 32 bits and grouped."""
    r = _rms(x)
    unit, g = x * r, dy * weight
    return r * (g - unit * (g * unit).mean(2, keepdim=True)), (dy * unit).sum((0, 3)).view(-1)


def _norm_bwd(s):
    dx, dw = _norm_grad(_grouped(s["x"], s), _channels(s["weight"], s), _grouped(s["dy"], s))
    return {"dx": (dx + _grouped(s["dres"], s)).view(_shape(s)).to(s["x"].dtype), "dweight": dw}


def _gate(s):
    """act(z) and its derivative, grouped; 1 and 0 without a gate."""
    if s["gate"] == "none":
        return 1.0, 0.0
    z = s["z"].float()
    z = z.view(s["n"], s["groups"], s["c"] // s["groups"], -1)
    if s["act"] == "none":
        return z, torch.ones_like(z)
    sig = 1.0 / (1.0 + torch.exp(-z))
    if s["act"] == "sigmoid":
        return sig, sig * (1.0 - sig)
    return z * sig, sig * (1.0 + z * (1.0 - sig))


def _join_fwd(s):
    h, res = _grouped(s["h_"], s), _grouped(s["res"], s)
    a, _ = _gate(s)
    out = res + _channels(s["scale"], s) * a * (h * _rms(h) * _channels(s["weight"], s))
    nxt = out * _rms(out) * _channels(s["next_weight"], s)
    dt = s["res"].dtype
    return {"out": out.view(_shape(s)).to(dt), "next": nxt.view(_shape(s)).to(dt)}


def _join_bwd(s):
    out, h, dt = _grouped(s["res"], s), _grouped(s["h_"], s), s["res"].dtype
    w, k = _channels(s["weight"], s), _channels(s["scale"], s)
    a, da = _gate(s)
    dx, dnw = _norm_grad(out, _channels(s["next_weight"], s), _grouped(s["dnext"], s))
    dx = dx + _grouped(s["dout"], s)
    unit = h * _rms(h)
    dh, dwk = _norm_grad(h, w, dx * k * a)
    res = {"dres": dx.view(_shape(s)).to(dt), "dh": dh.view(_shape(s)).to(dt), "dweight": dwk,
           "dscale": (dx * a * unit * w).sum((0, 3)).view(-1), "dnext_weight": dnw}
    if s["gate"] == "full":
        res["dgate"] = (dx * k * w * unit * da).view(_shape(s)).to(dt)
    elif s["gate"] == "channel":
        res["dgate"] = (dx * k * w * unit * da).sum(3).view(s["n"], s["c"])
    return res


def _matrices(t, s):
    return t.float().view(s["groups"], s["co"] // s["groups"], -1)


def _orth(x):
    a, b, c = NS
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(STEPS):
        gram = x @ x.mT
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.mT if tall else x


def _orth_plain(s):
    return {"out": _orth(_matrices(s["g"], s)).reshape(s["g"].shape).to(torch.bfloat16)}


def _scale(s):
    rows, cols = s["co"] // s["groups"], s["ci"] // s["groups"] * s["kh"] * s["kw"]
    return math.sqrt(max(1.0, rows / cols))


def _muon_plain(s):
    m = BETA * s["m"] + s["g"]
    o = _orth(_matrices(s["g"] + BETA * m, s)).reshape(m.shape)
    w = s["w"] * (1.0 - LR * DECAY) - (LR * _scale(s)) * o
    return {"w": w, "m": m, "w_bf16": w.to(torch.bfloat16)}


_PLAIN = {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "join_fwd": _join_fwd, "join_bwd": _join_bwd,
          "orth": _orth_plain, "muon": _muon_plain}


def run(s):
    if not own:
        return _PLAIN[s["op"]](s)
    import bwd_gconv_fwd_gb300 as gc
    op, groups = s["op"], s["groups"]
    if op == "norm_fwd":
        gc.gconv_norm_fwd(s["x"], s["weight"], s["y"], groups=groups, eps=EPS)
        return {"y": s["y"]}
    if op == "norm_bwd":
        gc.gconv_norm_bwd(s["x"], s["weight"], s["dy"], s["dx"], s["dweight"], dres=s["dres"], groups=groups, eps=EPS)
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "join_fwd":
        gc.gconv_join_fwd(s["res"], s["h_"], s["out"], gate=s["z"], act=s["act"], weight=s["weight"], scale=s["scale"],
                          next=s["next"], next_weight=s["next_weight"], groups=groups, eps=EPS)
        return {"out": s["out"], "next": s["next"]}
    if op == "join_bwd":
        gc.gconv_join_bwd(s["h_"], s["dout"], s["dh"], gate=s["z"], act=s["act"], weight=s["weight"], scale=s["scale"],
                          dgate=s["dz"], dweight=s["dweight"], dscale=s["dscale"],
                          out=s["res"], next_weight=s["next_weight"], dnext=s["dnext"], dres=s["dres"],
                          dnext_weight=s["dnext_weight"], groups=groups, eps=EPS)
        got = {"dres": s["dres"], "dh": s["dh"], "dweight": s["dweight"], "dscale": s["dscale"],
               "dnext_weight": s["dnext_weight"]}
        if s["dz"] is not None:
            got["dgate"] = s["dz"]
        return got
    if op == "orth":
        gc.gconv_orthogonalize(s["g"], s["out"], groups=groups, steps=STEPS, coeffs=NS, eps=NS_EPS)
        return {"out": s["out"]}
    gc.gconv_muon_step(s["w"], s["g"], s["m"], w_out=s["w_out"], m_out=s["m_out"], w_bf16=s["w_bf16"], groups=groups,
                       lr=LR, beta=BETA, weight_decay=DECAY, nesterov=True, steps=STEPS, coeffs=NS, eps=NS_EPS)
    return {"w": s["w_out"], "m": s["m_out"], "w_bf16": s["w_bf16"]}


# ---- the definitions in 64 bits ---------------------------------------------------


def _exact_unit(t, weight, groups):
    """t / sqrt(mean of squares + eps) * weight, channel block by channel block."""
    n, c = t.shape[:2]
    power = torch.einsum("ngkhw,ngkhw->nghw", *(2 * [t.reshape(n, groups, c // groups, *t.shape[2:])])) / (c // groups)
    size = torch.sqrt(power + EPS).repeat_interleave(c // groups, 1)
    return t / size * weight[:, None, None]


def _exact_orth(g):
    """Q g / |g| with Q gathered on the small side: every factor is a polynomial in one Gram matrix."""
    a, b, c = NS
    if g.shape[0] > g.shape[1]:
        return _exact_orth(g.t()).t()
    g = g / (torch.linalg.norm(g) + NS_EPS)
    gram = torch.einsum("ik,jk->ij", g, g)
    eye = torch.eye(g.shape[0], dtype=g.dtype, device=g.device)
    q = eye
    for _ in range(STEPS):
        p = a * eye + gram @ (b * eye + c * gram)
        q, gram = p @ q, p @ gram @ p
    return q @ g


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op, groups = case["op"], case["groups"]
    if op == "norm_fwd":
        return {"y": _exact_unit(d["x"], d["weight"], groups)}
    if op in ("orth", "muon"):
        u = d["g"]
        if op == "muon":
            beta = BETA
            m = d["m"] * beta + d["g"]
            u = d["g"] + m * beta
        o = torch.cat([_exact_orth(x.reshape(x.shape[0], -1)) for x in u.chunk(groups, 0)]).reshape(u.shape)
        if op == "orth":
            return {"out": o}
        w = d["w"] - LR * DECAY * d["w"] - LR * _scale(s) * o
        return {"w": w, "m": m, "w_bf16": w}
    act = {"none": lambda z: z, "sigmoid": torch.sigmoid, "silu": lambda z: z * torch.sigmoid(z)}[case["act"]]

    def branch(v):
        z = 1.0 if case["gate"] == "none" else act(v["z"])
        z = z[:, :, None, None] if case["gate"] == "channel" else z
        return v["scale"][:, None, None] * z * _exact_unit(v["h_"], v["weight"], groups)

    if op == "join_fwd":
        out = d["res"] + branch(d)
        return {"out": out, "next": _exact_unit(out, d["next_weight"], groups)}

    def grads(f, names, dy):
        v = dict(d, **{k: d[k].requires_grad_() for k in names})
        return torch.autograd.grad(f(v), [v[k] for k in names], dy)

    if op == "norm_bwd":
        dx, dw = grads(lambda v: _exact_unit(v["x"], v["weight"], groups), ("x", "weight"), d["dy"])
        return {"dx": dx + d["dres"], "dweight": dw}
    dx, dnw = grads(lambda v: _exact_unit(v["res"], v["next_weight"], groups), ("res", "next_weight"), d["dnext"])
    dx = (dx + d["dout"]).detach()
    names = ["h_", "weight", "scale"] + (["z"] if case["gate"] != "none" else [])
    got = grads(branch, names, dx)
    res = {"dres": dx, "dh": got[0], "dweight": got[1], "dscale": got[2], "dnext_weight": dnw}
    if case["gate"] != "none":
        res["dgate"] = got[3]
    return res


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("orth", "muon"):
        rows, cols = case["co"] // case["groups"], case["ci"] // case["groups"] * case["kh"] * case["kw"]
        m, n, e = min(rows, cols), max(rows, cols), case["groups"] * rows * cols
        # the Gram matrix and its square are symmetric: half of each
        flops = case["groups"] * STEPS * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)
        return {"bytes": e * (b + 2 if case["op"] == "orth" else 22), "flops": flops}
    e = case["n"] * case["c"] * case["h"] * case["w"]
    full = case["gate"] == "full"
    streams = {"norm_fwd": 2, "norm_bwd": 4, "join_fwd": 4 + full, "join_bwd": 6 + 2 * full}[case["op"]]
    ops = {"norm_fwd": 4, "norm_bwd": 12, "join_fwd": 12, "join_bwd": 30}[case["op"]]
    vectors = {"norm_fwd": 1, "norm_bwd": 2, "join_fwd": 3, "join_bwd": 6}[case["op"]]
    gates = case["n"] * case["c"] * (b + 4 * (case["op"] == "join_bwd")) if case["gate"] == "channel" else 0
    return {"bytes": streams * e * b + 4 * vectors * case["c"] + gates, "flops": ops * e}
