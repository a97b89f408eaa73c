"""The causal convolution, selective scan and dropout cases that are timed and checked.

Layout is the library's: activations [N, C, L], a sequence being a plane whose L positions follow one another.  Group g of
`groups` owns C/groups consecutive channels, which share S channels of B and of C.

  causal   y[t] = act(bias + sum_k w[k] x[t - K + 1 + k]),  x before position 0 from `state` [N, C, K-1]
  scan     d = softplus(delta + delta_bias),  h[t] = exp(d A) h[t-1] + d B[t] u[t]  for each of S states,
           y = (sum_s C[t] h[t] + D u) silu(z);  h before position 0 from `state` [N, C, S]
  dropout  y = res + keep x / (1 - p);  keep[e] = word e % 4 of Philox-4x32-10 (Salmon et al., 2011) at the
           counter (e / 4, step) under the key seed is at least p 2^32;  rng holds (seed, step)

A sequence of `lengths[n]` positions shorter than L has zeros behind them, in results and in gradients.
"""
import math

import torch

own = False

KEYS = (0x9E3779B9, 0xBB67AE85)
FACTORS = (0xD2511F53, 0xCD9E8D57)
LOW = 0xFFFFFFFF


def _causal(name, op, dtype, n, c, l, k, act, ragged=False, carried=False):
    case = {"op": op, "dtype": dtype, "n": n, "c": c, "l": l, "k": k, "act": act, "ragged": ragged, "carried": carried}
    return dict(case, name=name) if name else case


def _scan(name, op, dtype, n, c, l, s, groups, gated, ragged=False, carried=False):
    case = {"op": op, "dtype": dtype, "n": n, "c": c, "l": l, "s": s, "groups": groups, "gated": gated, "ragged": ragged,
            "carried": carried}
    return dict(case, name=name) if name else case


def _drop(name, op, dtype, shape, p, res):
    case = {"op": op, "dtype": dtype, "n": shape[0], "c": shape[1], "h": shape[2], "w": shape[3], "p": p, "res": res}
    return dict(case, name=name) if name else case


def listed():
    return [
        # one new position of eight sequences: latency
        _causal("causal_token", "causal_fwd", "bf16", 8, 1024, 1, 4, "silu", carried=True),
        # a training batch of a wide layer
        _causal("causal_fwd", "causal_fwd", "bf16", 8, 2048, 2048, 4, "silu"),
        _causal("causal_bwd", "causal_bwd", "bf16", 8, 2048, 2048, 4, "silu"),
        # fp32, rows never aligned, sequences of unlike lengths
        _causal("causal_bwd_ragged_f32", "causal_bwd", "f32", 7, 512, 1023, 4, "silu", ragged=True),
        # one new position of 64 sequences
        _scan("scan_token", "scan_fwd", "bf16", 64, 2048, 1, 16, 1, True, carried=True),
        # a prompt of one sequence, whose state goes on to the single positions
        _scan("scan_prompt", "scan_fwd", "bf16", 1, 2048, 4096, 16, 1, True, carried=True),
        # a long sequence of few channels: work only along the positions
        _scan("scan_long", "scan_fwd", "bf16", 1, 256, 65536, 16, 1, False),
        # the fp32 layer of five groups of 20 channels, 28 x 28 positions, sequences of unlike lengths
        _scan("scan_train_g5_f32", "scan_train", "f32", 8, 100, 784, 16, 5, False, ragged=True),
        # a training batch: forward and backward
        _scan("scan_train", "scan_train", "bf16", 8, 2048, 2048, 16, 1, True),
        # the fp32 layer's activations: smallest
        _drop("dropout_tiny_f32", "dropout_fwd", "f32", (2, 100, 28, 28), 0.5, False),
        # a large bottleneck stage's branch joining the residual, and its gradient
        _drop("dropout_56x56", "dropout_fwd", "bf16", (64, 256, 56, 56), 0.1, True),
        _drop("dropout_bwd_56x56", "dropout_bwd", "bf16", (64, 256, 56, 56), 0.1, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["causal_fwd", "causal_bwd", "scan_fwd", "scan_fwd", "scan_train", "scan_train", "dropout_fwd",
                     "dropout_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = 33_000_000 if dtype == "bf16" else 16_000_000
    if op.startswith("dropout"):
        h = rng.choice([1, 7, 13, 14, 27, 28, 56])
        c = _log(rng, 1, 2048)
        n = max(1, min(_log(rng, 1, 256), most // (c * h * h)))
        return _drop(None, op, dtype, (n, c, h, h), rng.choice([0.05, 0.1, 0.25, 0.5]), op == "dropout_fwd" and rng.random() < 0.5)
    ragged, carried = rng.random() < 0.3, rng.random() < 0.4
    if op.startswith("causal"):
        c = _log(rng, 16, 4096)
        l = rng.choice([1, _log(rng, 2, 8192), _log(rng, 2, 8192), 8 * _log(rng, 1, 1024)])
        n = max(1, min(_log(rng, 1, 64), most // (c * l)))
        return _causal(None, op, dtype, n, c, l, rng.choice([2, 3, 4, 4]), rng.choice(["silu", "silu", "none"]), ragged, carried)
    groups = rng.choice([1, 1, 1, 2, 5])
    s = rng.choice([4, 8, 16, 16, 16, 24, 64])
    c = _log(rng, 16, 2048 // groups) * groups
    longest = 32768 if op == "scan_fwd" else 4096
    l = rng.choice([1 if op == "scan_fwd" else 64, _log(rng, 2, longest), _log(rng, 2, longest), 8 * _log(rng, 1, longest // 8)])
    most = most * 16 // s
    l = min(l, max(1, most // c))
    n = max(1, min(_log(rng, 1, 64), most // (c * l)))
    return _scan(None, op, dtype, n, c, l, s, groups, rng.random() < 0.5, ragged, carried)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(case):
    return [case["l"] - i * case["l"] // case["n"] for i in range(case["n"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _dtype(case)
    op = case["op"]

    def normal(shape, sd=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, device=dev).normal_(mean, sd, generator=gen).to(dtype)

    new = lambda shape, d=dt: torch.empty(shape, device=dev, dtype=d)  # noqa: E731
    s = dict(case)
    n, c = case["n"], case["c"]
    if op.startswith("dropout"):
        shape = (n, c, case["h"], case["w"])
        s["x"] = normal(shape, dtype=dt)
        s["r"] = normal(shape, 2.0, dtype=dt) if case["res"] else None
        s["rng"] = torch.tensor([int(seed) * 7919 + 13, 1000 + int(seed) % 17], dtype=torch.int64, device=dev)
        s["y"] = new(shape)
        return s
    shape = (n, c, case["l"])
    s["lengths"] = None
    if case["ragged"]:
        order = torch.rand((n,), device=dev, generator=gen).argsort()
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[order].contiguous()
    if op.startswith("causal"):
        k = case["k"]
        s["x"] = normal(shape, dtype=dt)
        s["weight"], s["bias"] = normal((c, k), k ** -0.5), normal((c,), 0.1)
        s["state"] = normal((n, c, k - 1), dtype=dt) if case["carried"] else None
        s["state_out"] = new((n, c, k - 1)) if case["carried"] and op == "causal_fwd" else None
        if op == "causal_fwd":
            s["y"] = new(shape)
        else:
            s["dy"] = normal(shape, dtype=dt)
            s["dx"], s["dw"], s["db"] = new(shape), new((c, k), torch.float32), new((c,), torch.float32)
            s["dstate"] = new((n, c, k - 1)) if case["carried"] else None
        return s
    states, groups = case["s"], case["groups"]
    # u follows a silu; steps d between 0.001 and 0.1, log-uniform over the channels, moved by delta; decays -1 to -S
    u = normal(shape)
    s["u"] = (u * torch.sigmoid(u)).to(dt)
    s["delta"] = normal(shape, 0.4, dtype=dt)
    step = torch.exp(torch.rand((c,), device=dev, generator=gen) * math.log(100.0) + math.log(0.001))
    s["delta_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, states + 1, device=dev, dtype=torch.float32) * torch.exp(normal((c, states), 0.1))
    s["B"], s["C"] = normal((n, groups * states, case["l"]), dtype=dt), normal((n, groups * states, case["l"]), dtype=dt)
    s["D"] = normal((c,), 0.1, 1.0)
    s["z"] = normal(shape, dtype=dt) if case["gated"] else None
    s["state"] = normal((n, c, states), 0.5) if case["carried"] else None
    s["state_out"] = new((n, c, states), torch.float32) if case["carried"] else None
    s["y"] = new(shape)
    if op == "scan_train":
        s["dy"] = normal(shape, dtype=dt)
        s["du"], s["ddelta"], s["dz"] = new(shape), new(shape), new(shape) if case["gated"] else None
        s["dB"], s["dC"] = new(s["B"].shape), new(s["B"].shape)
        s["dA"] = new((c, states), torch.float32)
        s["dD"], s["ddelta_bias"] = new((c,), torch.float32), new((c,), torch.float32)
        s["dstate"] = new((n, c, states), torch.float32) if case["carried"] else None
        s["saved"] = None
        if own:
            import bwd_gconv_fwd_gb300 as gc
            size = gc.gconv_scan_saved_size(shape, states, gc.GCONV_BF16 if dt == torch.bfloat16 else gc.GCONV_F32,
                                            gated=case["gated"])
            s["saved"] = torch.empty(size, dtype=torch.uint8, device=dev)
    return s


# ---- the plain forms ------------------------------------------------------------


def _valid(s):
    """[N, 1, L]: whether a position is one of its sequence."""
    at = torch.arange(s["l"], device="cuda")
    if s["lengths"] is None:
        return torch.ones((s["n"], 1, s["l"]), dtype=torch.bool, device="cuda")
    return (at < s["lengths"][:, None])[:, None]


def _windows(s, ok):
    """x behind its state, zeros outside the sequence: [N, C, K - 1 + L]."""
    x = torch.where(ok, s["x"].float(), 0.0)
    head = torch.zeros((s["n"], s["c"], s["k"] - 1), device="cuda") if s["state"] is None else s["state"].float()
    return torch.cat([head, x], 2)


def _pre(s, x):
    v = s["bias"][:, None].expand(s["n"], s["c"], s["l"])
    for j in range(s["k"]):
        v = v + s["weight"][:, j, None] * x[:, :, j:j + s["l"]]
    return v


def _causal_fwd(s):
    ok = _valid(s)
    x = _windows(s, ok)
    v = _pre(s, x)
    if s["act"] == "silu":
        v = v / (1.0 + torch.exp(-v))
    got = {"y": torch.where(ok, v, 0.0).to(s["x"].dtype)}
    if s["state_out"] is not None:
        first = torch.full((s["n"],), s["l"], device="cuda") if s["lengths"] is None else s["lengths"].long()
        at = first[:, None, None] + torch.arange(s["k"] - 1, device="cuda")
        got["state"] = x.gather(2, at.expand(s["n"], s["c"], s["k"] - 1)).to(s["x"].dtype)
    return got


def _causal_bwd(s):
    ok = _valid(s)
    x = _windows(s, ok)
    dv = torch.where(ok, s["dy"].float(), 0.0)
    if s["act"] == "silu":
        v = _pre(s, x)
        sig = 1.0 / (1.0 + torch.exp(-v))
        dv = dv * sig * (1.0 + v * (1.0 - sig))
    k, l = s["k"], s["l"]
    none = torch.zeros((s["n"], s["c"], k - 1), device="cuda")
    wide = torch.cat([none, dv, none], 2)
    dx = sum(s["weight"][:, j, None] * wide[:, :, k - 1 - j:2 * k - 2 - j + l] for j in range(k))
    dw = torch.stack([(dv * x[:, :, j:j + l]).sum((0, 2)) for j in range(k)], 1)
    got = {"dx": torch.where(ok, dx[:, :, k - 1:], 0.0).to(s["x"].dtype), "dw": dw, "db": dv.sum((0, 2))}
    if s["dstate"] is not None:
        got["dstate"] = dx[:, :, :k - 1].to(s["x"].dtype)
    return got


def _recur(a, b):
    """h[t] = a[t] h[t-1] + b[t] along the last axis, by doubling; a and b are overwritten."""
    d = 1
    while d < a.shape[-1]:
        b[..., d:] = b[..., d:] + a[..., d:] * b[..., :-d]
        a[..., d:] = a[..., d:] * a[..., :-d]
        d *= 2
    return b


def _scan_plain(s, train):
    n, c, l, S, groups = s["n"], s["c"], s["l"], s["s"], s["groups"]
    cg = c // groups
    ok = _valid(s)
    dt = s["u"].dtype
    u = torch.where(ok, s["u"].float(), 0.0)
    t = s["delta"].float() + s["delta_bias"][:, None]
    d = torch.where(ok, t.clamp(min=0.0) + torch.log1p(torch.exp(-t.abs())), 0.0)
    gate = dgate = None
    if s["z"] is not None:
        z = torch.where(ok, s["z"].float(), 0.0)
        sig = 1.0 / (1.0 + torch.exp(-z))
        gate, dgate = z * sig, sig * (1.0 + z * (1.0 - sig))
    y = torch.empty((n, c, l), device="cuda")
    last, origin = torch.empty((n, c, S), device="cuda"), torch.empty((n, c, S), device="cuda")
    Bm, Cm = (torch.where(ok[:, :, None], m.float().view(n, groups, S, l), 0.0) for m in (s["B"], s["C"]))
    if train:
        dout = torch.where(ok, s["dy"].float(), 0.0)
        dy = dout if gate is None else dout * gate
        du, dd, dA = torch.empty_like(u), torch.empty_like(u), torch.empty((c, S), device="cuda")
        dB, dC = torch.zeros((n, groups, S, l), device="cuda"), torch.zeros((n, groups, S, l), device="cuda")
    some = max(1, (1 << 27) // (n * S * l))     # channels at once
    for g in range(groups):
        Bg, Cg = Bm[:, g, None], Cm[:, g, None]
        for c0 in range(g * cg, (g + 1) * cg, some):
            at = slice(c0, min(c0 + some, (g + 1) * cg))
            A, dc, uc = s["A"][at, :, None], d[:, at, None], u[:, at, None]
            b = (dc * uc) * Bg
            a = torch.exp(dc * A)
            first = torch.zeros((n, b.shape[1], S), device="cuda") if s["state"] is None else s["state"][:, at]
            b[..., 0] += a[..., 0] * first
            h = _recur(a, b)
            y[:, at] = (Cg * h).sum(2)
            last[:, at] = h[..., -1]
            if not train:
                continue
            a = torch.exp(dc * A)
            after = torch.zeros_like(a)
            after[..., :-1] = a[..., 1:]
            dh = (_recur(after.flip(-1), (dy[:, at, None] * Cg).flip(-1))).flip(-1)
            dC[:, g] += (dy[:, at, None] * h).sum(1)
            dB[:, g] += (dh * (dc * uc)).sum(1)
            q = a * torch.cat([first[..., None], h[..., :-1]], 3) * dh
            dA[at] = (q * dc).sum((0, 3))
            origin[:, at] = a[..., 0] * dh[..., 0]
            sb = (dh * Bg).sum(2)
            du[:, at] = d[:, at] * sb
            dd[:, at] = u[:, at] * sb + (q * A).sum(2)
    pre = y + s["D"][:, None] * u
    got = {"y": torch.where(ok, pre if gate is None else pre * gate, 0.0).to(dt)}
    if s["state_out"] is not None:
        got["state"] = last
    if train:
        dd = dd / (1.0 + torch.exp(-t))
        dd = torch.where(ok, dd, 0.0)
        got["du"] = (du + s["D"][:, None] * dy).to(dt)
        got["ddelta"], got["ddelta_bias"] = dd.to(dt), dd.sum((0, 2))
        got["dA"], got["dD"] = dA, (dy * u).sum((0, 2))
        got["dB"], got["dC"] = dB.view(n, -1, l).to(dt), dC.view(n, -1, l).to(dt)
        if gate is not None:
            got["dz"] = (dout * pre * dgate).to(dt)
        if s["dstate"] is not None:
            got["dstate"] = origin
    return got


def _keep(s):
    """Whether each element is kept, from its number and rng."""
    count = s["x"].numel()
    i = torch.arange((count + 3) // 4, device="cuda")
    seed, step = s["rng"][0], s["rng"][1]
    w = [i & LOW, i >> 32, (step & LOW).expand_as(i), ((step >> 32) & LOW).expand_as(i)]
    key = [seed & LOW, (seed >> 32) & LOW]
    for _ in range(10):
        p, q = w[0] * FACTORS[0], w[2] * FACTORS[1]      # 64 bits, which wrap
        w = [((q >> 32) & LOW) ^ w[1] ^ key[0], q & LOW, ((p >> 32) & LOW) ^ w[3] ^ key[1], p & LOW]
        key = [(key[0] + KEYS[0]) & LOW, (key[1] + KEYS[1]) & LOW]
    words = torch.stack(w, 1).view(-1)[:count].view(s["x"].shape)
    return words >= int(s["p"] * 2.0 ** 32)


def _dropout(s):
    bound = int(s["p"] * 2.0 ** 32)
    y = torch.where(_keep(s), s["x"].float() * (2.0 ** 32 / (2.0 ** 32 - bound)), 0.0)
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(s["x"].dtype)}


def run(s):
    op = s["op"]
    if not own:
        if op == "causal_fwd":
            return _causal_fwd(s)
        if op == "causal_bwd":
            return _causal_bwd(s)
        if op.startswith("scan"):
            return _scan_plain(s, op == "scan_train")
        return _dropout(s)
    import bwd_gconv_fwd_gb300 as gc
    if op == "causal_fwd":
        gc.gconv_causal_fwd(s["x"], s["weight"], s["bias"], s["y"], act=s["act"], state=s["state"], state_out=s["state_out"],
                            lengths=s["lengths"])
        return {"y": s["y"]} if s["state_out"] is None else {"y": s["y"], "state": s["state_out"]}
    if op == "causal_bwd":
        gc.gconv_causal_bwd(s["x"], s["weight"], s["bias"], s["dy"], s["dx"], s["dw"], s["db"], act=s["act"], state=s["state"],
                            lengths=s["lengths"], dstate=s["dstate"])
        got = {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
        return got if s["dstate"] is None else dict(got, dstate=s["dstate"])
    if op == "dropout_fwd":
        gc.gconv_dropout_fwd(s["x"], s["y"], s["rng"], s["p"], res=s["r"])
        return {"y": s["y"]}
    if op == "dropout_bwd":
        gc.gconv_dropout_bwd(s["x"], s["y"], s["rng"], s["p"])
        return {"y": s["y"]}
    gc.gconv_scan_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["y"], D=s["D"], z=s["z"], delta_bias=s["delta_bias"],
                      softplus=True, groups=s["groups"], state=s["state"], state_out=s["state_out"], lengths=s["lengths"],
                      saved=s.get("saved"))
    got = {"y": s["y"]}
    if s["state_out"] is not None:
        got["state"] = s["state_out"]
    if op == "scan_train":
        gc.gconv_scan_bwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["dy"], s["saved"], s["du"], s["ddelta"], s["dA"],
                          s["dB"], s["dC"], D=s["D"], z=s["z"], delta_bias=s["delta_bias"], softplus=True, groups=s["groups"],
                          lengths=s["lengths"], dD=s["dD"], dz=s["dz"], ddelta_bias=s["ddelta_bias"], dstate=s["dstate"])
        got.update({k: s[k] for k in ("du", "ddelta", "dA", "dB", "dC", "dD", "ddelta_bias")})
        got.update({k: s[k] for k in ("dz", "dstate") if s[k] is not None})
    return got


# ---- the definitions in 64 bits ---------------------------------------------------


def _counts(s):
    return [s["l"]] * s["n"] if s["lengths"] is None else s["lengths"].tolist()


def _exact_causal(s):
    """One sequence after another, cut to its own length."""
    f = {"none": lambda v: v, "silu": lambda v: v * torch.sigmoid(v)}[s["act"]]
    w, bias, k = s["weight"].double(), s["bias"].double(), s["k"]
    grad = s["op"] == "causal_bwd"
    full = torch.zeros((s["n"], s["c"], s["l"]), dtype=torch.float64, device="cuda")
    state = torch.zeros((s["n"], s["c"], k - 1), dtype=torch.float64, device="cuda")
    dw, db, dstate = torch.zeros_like(w), torch.zeros_like(bias), torch.zeros_like(state)
    for i, m in enumerate(_counts(s)):
        x = s["x"][i, :, :m].double()
        head = torch.zeros_like(state[i]) if s["state"] is None else s["state"][i].double()
        line = torch.cat([head, x], 1)
        state[i] = line[:, m:]
        if m == 0:
            continue
        taps = line.unfold(1, k, 1)
        v = torch.einsum("clk,ck->cl", taps, w) + bias[:, None]
        if not grad:
            full[i, :, :m] = f(v)
            continue
        sig = torch.sigmoid(v)
        dv = s["dy"][i, :, :m].double()
        if s["act"] == "silu":
            dv = dv * (sig + v * sig * (1 - sig))
        dw += torch.einsum("cl,clk->ck", dv, taps)
        db += dv.sum(1)
        pad = torch.cat([torch.zeros_like(head), dv, torch.zeros_like(head)], 1).unfold(1, k, 1)
        dline = torch.einsum("clk,ck->cl", pad, w.flip(1))
        dstate[i], full[i, :, :m] = dline[:, :k - 1], dline[:, k - 1:]
    if grad:
        got = {"dx": full, "dw": dw, "db": db}
        return got if s["dstate"] is None else dict(got, dstate=dstate)
    return {"y": full} if s["state_out"] is None else {"y": full, "state": state}


def _exact_scan(s):
    """Position after position."""
    n, c, l, S, groups = s["n"], s["c"], s["l"], s["s"], s["groups"]
    train = s["op"] == "scan_train"
    cg = c // groups
    there = torch.tensor(_counts(s), device="cuda")[:, None] > torch.arange(l, device="cuda")       # [N, L]
    first = lambda t: torch.where(there[:, None], t.double(), 0.0).permute(2, 0, 1).contiguous()  # noqa: E731  [L, N, ...]
    u, B, C = first(s["u"]), first(s["B"]).view(l, n, groups, 1, S), first(s["C"]).view(l, n, groups, 1, S)
    raw = first(s["delta"]) + s["delta_bias"].double()
    alive = there.t()[:, :, None]
    d = torch.where(alive, torch.logaddexp(raw, torch.zeros_like(raw)), 0.0)
    A = s["A"].double().view(groups, cg, S)
    h = torch.zeros((n, groups, cg, S), dtype=torch.float64, device="cuda")
    if s["state"] is not None:
        h = s["state"].double().view(h.shape)
    split = lambda t: t.view(n, groups, cg, 1)  # noqa: E731
    kept, y = [h], torch.zeros_like(u)
    for t in range(l):
        h = torch.exp(split(d[t]) * A) * h + split(d[t] * u[t]) * B[t]
        y[t] = (h * C[t]).sum(3).view(n, c)
        if train:
            kept.append(h)
    skip = s["D"].double()
    y += skip * u
    gate = pre = None
    if s["gated"]:
        z = first(s["z"])
        gate, pre = z * torch.sigmoid(z), y
        y = y * gate
    back = lambda t: t.permute(1, 2, 0)  # noqa: E731
    got = {"y": back(torch.where(alive, y, 0.0))}
    if s["state_out"] is not None:
        got["state"] = h.reshape(n, c, S)
    if not train:
        return got
    dout = first(s["dy"])
    dy = dout if gate is None else dout * gate
    if gate is not None:
        sig = torch.sigmoid(z)
        got["dz"] = back(dout * pre * (sig + z * sig * (1 - sig)))
    du, dd = skip * dy, torch.zeros_like(u)
    dB, dC = torch.zeros((l, n, groups, S), dtype=u.dtype, device="cuda"), torch.zeros((l, n, groups, S), dtype=u.dtype, device="cuda")
    dA = torch.zeros_like(A)
    g = torch.zeros_like(h)
    for t in range(l - 1, -1, -1):
        now = split(dy[t])
        g = g + now * C[t]
        dC[t] = (now * kept[t + 1]).sum(2)
        decay = torch.exp(split(d[t]) * A)
        p = g * decay * kept[t]
        dB[t] = (g * split(d[t] * u[t])).sum(2)
        gb = (g * B[t]).sum(3).view(n, c)
        du[t] += d[t] * gb
        dd[t] = u[t] * gb + (p * A).sum(3).view(n, c)
        dA += (p * split(d[t])).sum(0)
        g = g * decay
    dd = dd * torch.sigmoid(raw) * alive
    flat = lambda t: t.reshape(l, n, groups * S).permute(1, 2, 0)  # noqa: E731
    got.update(du=back(du), ddelta=back(dd), dA=dA.view(c, S), dB=flat(dB), dC=flat(dC), dD=(dy * u).sum((0, 1)),
               ddelta_bias=dd.sum((0, 1)))
    if s["dstate"] is not None:
        got["dstate"] = g.reshape(n, c, S)
    return got


def _product(a, b):
    """High and low word of the product of two 32-bit words, by halves of b."""
    high, low = a * (b >> 16), a * (b & 0xFFFF)
    return (high + (low >> 16)) >> 16, (((high & 0xFFFF) << 16) + low) & LOW


def _exact_dropout(s):
    seed, step = (int(v) & (2 ** 64 - 1) for v in s["rng"].tolist())
    count, flat = s["x"].numel(), s["x"].reshape(-1).double()
    bound = int(s["p"] * 2.0 ** 32)
    y = torch.zeros(count, dtype=torch.float64, device="cuda")
    block = torch.arange((count + 3) // 4, device="cuda")
    c0, c1, c2, c3 = block & LOW, block >> 32, torch.full_like(block, step & LOW), torch.full_like(block, step >> 32)
    for r in range(10):
        k0, k1 = ((seed & LOW) + r * KEYS[0]) & LOW, ((seed >> 32) + r * KEYS[1]) & LOW
        (h0, l0), (h1, l1) = _product(c0, FACTORS[0]), _product(c2, FACTORS[1])
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
    for j, word in enumerate((c0, c1, c2, c3)):
        part = flat[j::4]
        y[j::4] = part * (word[:part.numel()] >= bound).double() / (1.0 - bound / 2.0 ** 32)
    y = y.view(s["x"].shape)
    return {"y": y if s["r"] is None else y + s["r"].double()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("dropout"):
        return _exact_dropout(s)
    if case["op"].startswith("causal"):
        return _exact_causal(s)
    if case["op"] == "scan_train" and 8 * case["n"] * case["c"] * case["s"] * case["l"] > 40e9:
        return None
    return _exact_scan(s)


def work(case):
    b = 2 if case["dtype"] == "bf16" else 4
    op, n, c = case["op"], case["n"], case["c"]
    if op.startswith("dropout"):
        e = n * c * case["h"] * case["w"]
        return {"bytes": e * b * (3 if case["res"] else 2), "flops": 2 * e}
    at = sum(_lengths(case)) if case["ragged"] else n * case["l"]        # positions read
    e, full = at * c, n * c * case["l"]
    if op.startswith("causal"):
        k = case["k"]
        tail = n * c * (k - 1) * b * ((op == "causal_fwd") + 1) if case["carried"] else 0
        if op == "causal_fwd":
            return {"bytes": (e + full) * b + 4 * c * (k + 1) + tail, "flops": e * (2 * k + 5)}
        return {"bytes": (2 * e + full) * b + 8 * c * (k + 1) + tail, "flops": e * (6 * k + 12)}
    S = case["s"]
    gated = 1 if case["gated"] else 0
    small = 2 * at * case["groups"] * S * b + 4 * c * (S + 2) + (8 * n * c * S if case["carried"] else 0)
    fwd = {"bytes": ((2 + gated) * e + full) * b + small, "flops": e * (7 * S + 10)}
    if op == "scan_fwd":
        return fwd
    # backward: u, delta, dy, z read, du, ddelta, dz written; B, C read, dB, dC written
    more = ((3 + gated) * e + (2 + gated) * full) * b + 2 * small
    return {"bytes": fwd["bytes"] + more, "flops": fwd["flops"] + e * (22 * S + 20)}
