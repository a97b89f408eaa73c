"""Block norm and block join on the GPU against the definition in 64 bits.

Tolerances, from the arithmetic: a group's sums and r(t) are fp32 trees (relative error below
2^-24 times a few hundred terms a thread, about 1e-5 at worst), the exponential of the gate has
a relative error of a few 2^-22, so an fp32 result is within TOL = 2e-5 of the definition,
relative to the element plus the tensor's root mean square.  The norm's gradient is a difference,
r (g - u mean(g u)), that nearly vanishes in a group of one channel: there it is relative to
the root mean square of the term r g it starts from.  A bf16 result adds half a unit in the last place of 8 bits, 2^-8 of the
element at most.
"""
import numpy as np
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from bwd_gconv_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu

TOL = 2e-5
EPS = 1e-6
GUARD = 1024
ACT = {"none": lambda z: z, "sigmoid": torch.sigmoid, "silu": lambda z: z * torch.sigmoid(z)}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_gconv_fwd_gb300 import build
    build.build()
    return torch.device("cuda:0")


def unit(t, groups, eps=EPS):
    n, c, h, w = t.shape
    g = t.reshape(n, groups, c // groups, h, w)
    return (g / torch.sqrt((g * g).mean(2, keepdim=True) + eps)).reshape(t.shape)


def vec(v):
    return 1.0 if v is None else v[:, None, None]


def branch(h, gate, act, weight, scale, groups):
    z = 1.0
    if gate is not None:
        z = ACT[act](gate)
        z = z[:, :, None, None] if z.dim() == 2 else z
    return vec(scale) * z * unit(h, groups) * vec(weight)


def first_term(t, g, groups):
    """Root mean square of r(t) g."""
    n, c, h, w = t.shape
    m = t.double().reshape(n, groups, c // groups, h, w)
    r = 1 / torch.sqrt((m * m).mean(2, keepdim=True) + EPS)
    return (r * g.double().reshape(m.shape)).square().mean().sqrt().cpu()


def near(name, got, ref, dtype, size=None):
    g, r = got.double().cpu(), ref.double().cpu()
    rms = r.square().mean().sqrt() if size is None else size
    tol = TOL * (r.abs() + rms) + (2.0 ** -8 * r.abs() if dtype == torch.bfloat16 else 0.0)
    bad = (g - r).abs() > tol
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {r.numel()}, worst {float((g - r).abs().max()):.3e}, rms {float(rms):.3e}"


class Guarded:
    """Output tensors between guard words that must come back untouched."""

    def __init__(self, dev):
        self.dev, self.bufs = dev, []

    def __call__(self, shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((GUARD + n + GUARD,), float("nan"), device=self.dev, dtype=dtype)
        buf[:GUARD] = 7.5
        buf[GUARD + n:] = 7.5
        self.bufs.append((buf, n))
        return buf[GUARD:GUARD + n].view(shape)

    def check(self):
        for buf, n in self.bufs:
            assert bool((buf[:GUARD] == 7.5).all()) and bool((buf[GUARD + n:] == 7.5).all()), "write outside an output"


def make(shape, dtype, dev, seed, groups, gate="none"):
    gen = torch.Generator().manual_seed(seed)
    n, c = shape[:2]
    t = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {k: t(*shape).to(dtype).to(dev) for k in ("x", "h", "dout", "dnext")}
    d["gate"] = None if gate == "none" else (1.5 * t(*(shape if gate == "full" else shape[:2]))).to(dtype).to(dev)
    for k in ("weight", "scale", "next_weight"):
        d[k] = (1.0 + 0.3 * t(c)).to(dev)
    return d


def up(v):
    return None if v is None else v.double()


# (N, C, H, W, groups): one position, odd planes, planes of 2, 4 and 8 times an odd number, thin and
# wide groups, groups that take several thread blocks or are walked, several rows a block
SHAPES = [
    (1, 1, 1, 1, 1), (3, 8, 1, 1, 1), (2, 1000, 1, 1, 1), (5, 96, 1, 1, 2), (2, 5, 3, 3, 5), (2, 12, 1, 7, 4),
    (2, 100, 28, 28, 5), (3, 96, 27, 27, 2), (2, 48, 13, 13, 1), (1, 512, 7, 7, 1), (4, 128, 6, 4, 32), (2, 64, 14, 14, 1),
    (1, 256, 56, 56, 1), (2, 33, 2, 5, 1), (1, 2050, 4, 4, 1), (2, 4200, 1, 3, 1), (1, 9, 1, 4097, 3), (130, 16, 1, 2, 2),
    (1, 1536, 3, 8, 1), (2, 20, 5, 8, 1), (3, 1024, 7, 7, 1), (2, 2048, 7, 7, 1), (1, 3001, 5, 5, 1), (1, 40000, 1, 2, 1),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(dev, shape, dtype):
    *s, G = shape
    d = make(s, dtype, dev, 1, G)
    new = Guarded(dev)
    y, dx, dw = new(s, dtype), new(s, dtype), new((s[1],), torch.float32)
    gc.gconv_norm_fwd(d["x"], d["weight"], y, groups=G, eps=EPS)
    gc.gconv_norm_bwd(d["x"], d["weight"], d["dnext"], dx, dw, dres=d["dout"], groups=G, eps=EPS)
    x, w = up(d["x"]).requires_grad_(), up(d["weight"]).requires_grad_()
    ref = unit(x, G) * vec(w)
    near("y", y, ref.detach(), dtype)
    gx, gw = torch.autograd.grad(ref, (x, w), up(d["dnext"]))
    near("dx", dx, gx + up(d["dout"]), dtype, first_term(d["x"], up(d["dnext"]) * vec(up(d["weight"])), G))
    near("dweight", dw, gw, torch.float32)
    again = torch.empty_like(dw)
    gc.gconv_norm_bwd(d["x"], d["weight"], d["dnext"], dx, again, dres=d["dout"], groups=G, eps=EPS)
    assert torch.equal(again, dw)
    new.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate,act", [("none", "none"), ("full", "silu"), ("full", "none"), ("channel", "sigmoid"),
                                      ("channel", "silu"), ("full", "sigmoid")])
@pytest.mark.parametrize("shape", SHAPES)
def test_join(dev, shape, gate, act, dtype):
    *s, G = shape
    d = make(s, dtype, dev, 2, G, gate)
    new = Guarded(dev)
    out, nxt = new(s, dtype), new(s, dtype)
    kw = dict(gate=d["gate"], act=act, weight=d["weight"], scale=d["scale"], groups=G, eps=EPS)
    gc.gconv_join_fwd(d["x"], d["h"], out, next=nxt, next_weight=d["next_weight"], **kw)
    ref = up(d["x"]) + branch(up(d["h"]), up(d["gate"]), act, up(d["weight"]), up(d["scale"]), G)
    near("out", out, ref, dtype)
    near("next", nxt, unit(ref, G) * vec(up(d["next_weight"])), dtype)
    alone = new(s, dtype)
    gc.gconv_join_fwd(d["x"], d["h"], alone, **kw)
    assert torch.equal(alone, out)

    # the gradients at the stored out
    names = ["h", "weight", "scale"] + (["gate"] if gate != "none" else [])
    v = {k: up(d[k]) for k in names}
    for k in names:
        v[k].requires_grad_()
    f = branch(v["h"], v.get("gate"), act, v["weight"], v["scale"], G)
    o, nw = up(out).requires_grad_(), up(d["next_weight"]).requires_grad_()
    go, gnw = torch.autograd.grad(unit(o, G) * vec(nw), (o, nw), up(d["dnext"]))
    whole = go + up(d["dout"])
    for joined in (True, False):
        dh, dw, ds, dnw = new(s, dtype), new((s[1],), torch.float32), new((s[1],), torch.float32), new((s[1],), torch.float32)
        dres = new(s, dtype) if joined else None
        dg = None if gate == "none" else new(s, dtype) if gate == "full" else new(s[:2], torch.float32)
        more = dict(out=out, next_weight=d["next_weight"], dnext=d["dnext"], dres=dres, dnext_weight=dnw) if joined else {}
        gc.gconv_join_bwd(d["h"], d["dout"], dh, dgate=dg, dweight=dw, dscale=ds, **more, **kw)
        grads = torch.autograd.grad(f, [v[k] for k in names], whole if joined else up(d["dout"]), retain_graph=True)
        z = 1.0 if gate == "none" else ACT[act](up(d["gate"]))
        z = z[:, :, None, None] if gate == "channel" else z
        size = first_term(d["h"], (whole if joined else up(d["dout"])) * z * vec(up(d["weight"]) * up(d["scale"])), G)
        near("dh", dh, grads[0], dtype, size)
        near("dweight", dw, grads[1], torch.float32)
        near("dscale", ds, grads[2], torch.float32)
        if dg is not None:
            near("dgate", dg, grads[3], dg.dtype)
        if joined:
            near("dres", dres, whole, dtype, first_term(out, up(d["dnext"]) * vec(up(d["next_weight"])), G))
            near("dnext_weight", dnw, gnw, torch.float32)
    new.check()


# planes of one position: few and many rows, rows of a part of a warp up to several warps, wider than
# a block holds, groups, odd channels, groups shorter than a sector
ROWS = [
    (8, 1024, 1, 1, 1), (1000, 1024, 1, 1, 1), (700, 96, 1, 1, 2), (300, 33, 1, 1, 1), (2000, 64, 1, 1, 4), (3, 8192, 1, 1, 1),
    (2, 9000, 1, 1, 1), (65, 4100, 1, 1, 1), (1200, 21, 1, 1, 7), (333, 40, 1, 1, 5), (1, 16, 1, 1, 1), (400, 2056, 1, 1, 1),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", ROWS + [(1200, 7, 1, 1, 7)])
def test_norm_of_one_position(dev, shape, dtype):
    test_norm(dev, shape, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate,act", [("none", "none"), ("full", "silu"), ("channel", "sigmoid")])
@pytest.mark.parametrize("shape", ROWS)
def test_join_of_one_position(dev, shape, gate, act, dtype):
    test_join(dev, shape, gate, act, dtype)


# groups beyond a cluster's shared memory, in one type or both, of channel counts that do not divide into
# whole warps: planes of one tile, of a tile and a part, of many tiles, two groups
WALKED = [(1, 9001, 4, 4, 1), (2, 9001, 14, 14, 1), (1, 8193, 5, 5, 1), (3, 12345, 3, 3, 1), (1, 16401, 4, 4, 1),
          (2, 18014, 1, 7, 2), (1, 33001, 1, 2, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", WALKED)
def test_norm_of_wide_odd_groups(dev, shape, dtype):
    test_norm(dev, shape, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate,act", [("none", "none"), ("full", "silu"), ("channel", "sigmoid")])
@pytest.mark.parametrize("shape", WALKED)
def test_join_of_wide_odd_groups(dev, shape, gate, act, dtype):
    test_join(dev, shape, gate, act, dtype)


def test_rows_beside_the_last_add_nothing(dev):
    """eps = 0: r is infinite where a block has no row, which must not reach the channel sums."""
    s, G = (5, 64, 1, 1), 1
    d = make(s, torch.float32, dev, 9, G)
    dx, dw = torch.empty(s, device=dev), torch.empty(s[1], device=dev)
    gc.gconv_norm_bwd(d["x"], d["weight"], d["dnext"], dx, dw, groups=G, eps=0.0)
    near("dweight", dw, (up(d["dnext"]) * unit(up(d["x"]), G, 0.0)).sum((0, 2, 3)), torch.float32)


# one of each kernel family: rows, whole rows in shared memory, boxes, pieces, a cluster, walked groups
FAMILIES = [(9, 64, 1, 1, 1), (40, 66, 1, 1, 2), (3, 64, 7, 7, 1), (2, 64, 8, 16, 2), (2, 96, 27, 27, 2), (1, 1024, 14, 14, 1),
            (1, 16401, 4, 4, 1)]
# r(t)^3 alone leaves fp32 at each; the largest only where a group's squares stay in fp32 themselves
RANGES = [(1e-13, 0.0), (1e14, EPS), (1e16, EPS), (1e18, EPS)]


def far_apart(t, g, groups, eps):
    """Root mean square of r(t) g, as first_term, for any eps."""
    n, c, h, w = t.shape
    m = t.double().reshape(n, groups, c // groups, h, w)
    r = 1 / torch.sqrt((m * m).mean(2, keepdim=True) + eps)
    return (r * g.double().reshape(m.shape)).square().mean().sqrt().cpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size,eps", RANGES)
@pytest.mark.parametrize("shape", FAMILIES)
def test_gradients_of_small_and_large_activations(dev, shape, size, eps, dtype):
    *s, G = shape
    if size == 1e18 and s[1] // G > 64:
        pytest.skip("the sum of squares is beyond fp32")
    d = make(s, dtype, dev, 10, G)
    t = (d["x"].double() * size).to(dtype)
    dx, dw = torch.empty_like(t), torch.empty(s[1], device=dev)
    gc.gconv_norm_bwd(t, d["weight"], d["dnext"], dx, dw, groups=G, eps=eps)
    x, w = up(t).requires_grad_(), up(d["weight"]).requires_grad_()
    gx, gw = torch.autograd.grad(unit(x, G, eps) * vec(w), (x, w), up(d["dnext"]))
    near("dx", dx, gx, dtype, far_apart(t, up(d["dnext"]) * vec(up(d["weight"])), G, eps))
    near("dweight", dw, gw, torch.float32)
    dh, dw, ds = torch.empty_like(t), torch.empty(s[1], device=dev), torch.empty(s[1], device=dev)
    gc.gconv_join_bwd(t, d["dout"], dh, weight=d["weight"], scale=d["scale"], dweight=dw, dscale=ds, groups=G, eps=eps)
    k = up(d["weight"]) * up(d["scale"])
    gh, gw = torch.autograd.grad(unit(x, G, eps) * vec(w) * vec(up(d["scale"])), (x, w), up(d["dout"]))
    near("dh", dh, gh, dtype, far_apart(t, up(d["dout"]) * vec(k), G, eps))
    near("dweight", dw, gw, torch.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", FAMILIES)
def test_gradient_at_zeros_with_a_tiny_eps(dev, shape, dtype):
    """A position of zeros: the gradient is r g with r = 1 / sqrt(eps) = 1e15, whose cube is beyond fp32."""
    *s, G = shape
    d = make(s, dtype, dev, 11, G)
    x = d["x"].clone()
    x[0, :, 0, 0] = 0
    dx, dh = torch.empty_like(x), torch.empty_like(x)
    gc.gconv_norm_bwd(x, d["weight"], d["dnext"], dx, groups=G, eps=1e-30)
    near("dx at zeros", dx[0, :, 0, 0], up(d["dnext"])[0, :, 0, 0] * up(d["weight"]) * 1e15, dtype)
    gc.gconv_join_bwd(x, d["dout"], dh, weight=d["weight"], groups=G, eps=1e-30)
    near("dh at zeros", dh[0, :, 0, 0], up(d["dout"])[0, :, 0, 0] * up(d["weight"]) * 1e15, dtype)
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dh).all())


def test_join_without_vectors_or_dout(dev):
    """weight, scale and next_weight default to ones; dout may be missing beside dnext; the channel
    sums and dgate may be left out."""
    s, G = (2, 24, 5, 7), 3
    d = make(s, torch.float32, dev, 3, G, "full")
    out, nxt, dres, dh = (torch.empty(s, device=dev) for _ in range(4))
    gc.gconv_join_fwd(d["x"], d["h"], out, gate=d["gate"], act="silu", next=nxt, groups=G, eps=EPS)
    ref = up(d["x"]) + branch(up(d["h"]), up(d["gate"]), "silu", None, None, G)
    near("out", out, ref, torch.float32)
    near("next", nxt, unit(ref, G), torch.float32)
    gc.gconv_join_bwd(d["h"], None, dh, gate=d["gate"], act="silu", out=out, dnext=d["dnext"], dres=dres, groups=G, eps=EPS)
    o, h = up(out).requires_grad_(), up(d["h"]).requires_grad_()
    go, = torch.autograd.grad(unit(o, G), o, up(d["dnext"]))
    gh, = torch.autograd.grad(branch(h, up(d["gate"]), "silu", None, None, G), h, go)
    near("dres", dres, go, torch.float32)
    near("dh", dh, gh, torch.float32)


@pytest.mark.parametrize("gate", ["none", "full", "channel"])
def test_gradients_against_differences(dev, gate):
    """<gradient, v> against the central difference of the definition along v, in 64 bits."""
    s, G = (2, 18, 3, 5), 3
    d = make(s, torch.float32, dev, 4, G, gate)
    out, nxt, dres, dh = (torch.empty(s, device=dev) for _ in range(4))
    kw = dict(gate=d["gate"], act="silu", weight=d["weight"], scale=d["scale"], groups=G, eps=EPS)
    gc.gconv_join_fwd(d["x"], d["h"], out, next=nxt, next_weight=d["next_weight"], **kw)
    dg = None if gate == "none" else torch.empty_like(d["gate"])
    dw, ds, dnw = (torch.empty(s[1], device=dev) for _ in range(3))
    gc.gconv_join_bwd(d["h"], d["dout"], dh, dgate=dg, dweight=dw, dscale=ds, out=out, next_weight=d["next_weight"],
                      dnext=d["dnext"], dres=dres, dnext_weight=dnw, **kw)

    def loss(v):
        o = v["x"] + branch(v["h"], v["gate"], "silu", v["weight"], v["scale"], G)
        return float((o * up(d["dout"])).sum() + (unit(o, G) * vec(v["next_weight"]) * up(d["dnext"])).sum())

    gen = torch.Generator().manual_seed(5)
    for key, grad in (("x", dres), ("h", dh), ("gate", dg), ("weight", dw), ("scale", ds), ("next_weight", dnw)):
        if grad is None:
            continue
        base = {k: up(v) for k, v in d.items()}
        way = torch.randn(base[key].shape, generator=gen).double().to(dev)
        step = 1e-4
        diff = (loss(dict(base, **{key: base[key] + step * way})) - loss(dict(base, **{key: base[key] - step * way}))) / (2 * step)
        got = float((grad.double() * way).sum())
        # the difference is off by step^2 times a third derivative of order one; the gradient by
        # TOL of its root mean square an element, adding like a random walk
        size = float((grad.double() * way).norm())
        assert abs(got - diff) <= TOL * 4 * size + 1e-6 * (1 + abs(diff)), key


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zero_and_infinite_positions(dev, dtype):
    """A position of zeros has r = 1/sqrt(eps); a position with an Inf or NaN spoils its own group only."""
    s, G = (1, 8, 3, 3), 2
    d = make(s, dtype, dev, 6, G)
    x = d["x"].clone()
    x[0, :4, 0, 0] = 0
    x[0, 1, 1, 1] = float("inf")
    x[0, 6, 2, 2] = float("nan")
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(8, device=dev)
    gc.gconv_norm_fwd(x, d["weight"], y, groups=G, eps=EPS)
    ref = unit(up(x), G) * vec(up(d["weight"]))
    assert torch.equal(torch.isnan(y), torch.isnan(ref)) and torch.equal(torch.isinf(y), torch.isinf(ref))
    fine = torch.isfinite(ref)
    near("y", y[fine], ref[fine], dtype)
    assert int((~torch.isfinite(y)).sum()) == 5   # the Inf itself, and the NaN's group
    gc.gconv_norm_bwd(x, d["weight"], d["dnext"], dx, dw, groups=G, eps=EPS)
    r = EPS ** -0.5
    near("dx at zeros", dx[0, :4, 0, 0], up(d["dnext"])[0, :4, 0, 0] * up(d["weight"])[:4] * r, dtype)


def test_other_stream_and_given_workspace(dev):
    s, G = (4, 64, 14, 14), 2
    d = make(s, torch.bfloat16, dev, 7, G)
    need = gc.gconv_block_workspace_size(s, B.GCONV_BF16, G)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    want, got = [(torch.empty(s, device=dev, dtype=torch.bfloat16), torch.empty(64, device=dev)) for _ in range(2)]
    gc.gconv_norm_bwd(d["x"], d["weight"], d["dnext"], *want, groups=G)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    gc.gconv_norm_bwd(d["x"], d["weight"], d["dnext"], *got, groups=G, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    with pytest.raises(gc.GconvError):
        gc.gconv_norm_bwd(d["x"], d["weight"], d["dnext"], *got, groups=G, workspace=ws[:need - 1])


def test_empty_batch_and_refusals(dev):
    x, w = torch.empty((0, 8, 3, 3), device=dev), torch.ones(8, device=dev)
    dw = torch.full((8,), 3.0, device=dev)
    gc.gconv_norm_fwd(x, w, torch.empty_like(x))
    gc.gconv_norm_bwd(x, w, x, torch.empty_like(x), dw)
    assert bool((dw == 0).all())
    x = torch.ones((2, 8, 3, 3), device=dev)
    y = torch.empty_like(x)
    for bad in (lambda: gc.gconv_norm_fwd(x, w, y, groups=3),                       # channels not divisible
                lambda: gc.gconv_norm_fwd(x, w, y, eps=-1.0),
                lambda: gc.gconv_norm_fwd(x, w, y, eps=float("nan")),
                lambda: gc.gconv_norm_fwd(x.half(), w, y),
                lambda: gc.gconv_norm_fwd(x, w[:4], y),
                lambda: gc.gconv_norm_fwd(x, w, y.bfloat16()),
                lambda: gc.gconv_norm_fwd(x.transpose(2, 3)[:, :, :, :2], w, y[:, :, :, :2]),   # strides
                lambda: gc.gconv_norm_fwd(x.cpu(), w, y),
                lambda: gc.gconv_join_fwd(x, x, y, gate=w),
                lambda: gc.gconv_join_fwd(x, x, y, act="gelu"),
                lambda: gc.gconv_join_fwd(x, x, y, next_weight=w),                  # no next
                lambda: gc.gconv_join_bwd(x, None, y),                              # no gradient at all
                lambda: gc.gconv_join_bwd(x, x, y, dnext=x),                        # next without out, dres
                lambda: gc.gconv_join_bwd(x, x, y, dgate=y.clone()),                # no gate
                lambda: gc.gconv_join_bwd(x, x, y, gate=x[:, :, 0, 0].contiguous(), dgate=torch.empty_like(x))):
        with pytest.raises((gc.GconvError, ValueError, TypeError)):
            bad()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", FAMILIES + [(64, 128, 56, 56, 1), (32, 1024, 7, 7, 1)])
def test_wait_timeout_is_reported_and_recovered(dev, shape, dtype):
    """With a wait limit of zero a wait that is not over at its first poll gives up (a poll may itself last
    until the copies have landed, and some kernels have no such wait): the call then reports it, else its
    result is right, and either way the next call, with the limit restored, is right."""
    *s, G = shape
    d = make(s, dtype, dev, 12, G)
    call = lambda dx, dw: gc.gconv_norm_bwd(d["x"], d["weight"], d["dnext"], dx, dw, dres=d["dout"], groups=G)  # noqa: E731
    want, tried, got = ((torch.empty_like(d["x"]), torch.empty(s[1], device=dev)) for _ in range(3))
    call(*want)
    assert gc.gconv_check_device_error() == B.GCONV_OK
    B.gconv_debug_set_wait_limit(0)
    try:
        call(*tried)
        status = gc.gconv_check_device_error()
    finally:
        B.gconv_debug_set_wait_limit(-1)
    same = lambda a: all(torch.equal(u, v) for u, v in zip(a, want))  # noqa: E731
    assert status == B.GCONV_ERR_TIMEOUT or (status == B.GCONV_OK and same(tried))
    call(*got)
    assert gc.gconv_check_device_error() == B.GCONV_OK and same(got)
