"""The causal convolution and the selective scan on the GPU against their definitions in 64 bits.

Tolerances, from the arithmetic.  The scan's state is a sum over earlier positions whose weights are products of
decays.  A decay has a relative error of (1 + |d A|) times at most 2^-20: the base-2 exponential's approximation (2^-22), the
roundings of d, A log2 e and their product (|d A| 2^-22), the sums of d over a run (|d A| 2^-21).  So the error of a state is at
most 2^-20 times E, E[t] = exp(d A) (E[t-1] + (1 + |d A|) H[t-1]) + 2 |d u B|, where H is the state made of absolute values, and M = max E / H is
the number of roundings that a term has gone through.  Every result is such a sum, or (gradients) a sum over
products of two of them: an fp32 result is within 2^-20 (2 M + 8) of the same result made of absolute
values.  A bf16 result adds half a unit in the last place, 2^-8 of it; dz is made from a sum that was rounded to bf16 before, so
2^-7.  The convolution adds at most 8 products (2^-20 of the absolute sum with the sigmoid, whose
argument's rounding adds |v| 2^-22), its channel sums at most 2^9 terms one after the other (2^-15).
"""
import numpy as np
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from bwd_gconv_fwd_gb300 import binding as B_

pytestmark = pytest.mark.gpu
GUARD = 1024
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_gconv_fwd_gb300 import build
    build.build()
    return torch.device("cuda:0")


class Guarded:
    """Outputs between guard words that must come back untouched; NaN inside until they are written."""

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


def near(name, got, ref, mag, tol, dtype=F32, steps=1):
    """|got - ref| <= tol mag + the dtype's rounding of ref, `steps` times."""
    g, r = got.double(), ref
    bound = tol * mag + (steps * 2.0 ** -8 * r.abs() if dtype == BF16 else 2.0 ** -23 * r.abs()) + 1e-30
    bad = ~((g - r).abs() <= bound)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {r.numel()} off, worst {float(((g - r).abs() / bound).max()):.2f} bounds"


# ---- the scan --------------------------------------------------------------------


def scan_ref(d, dy=None, dstate_out=None, size=False):
    """Position after position in 64 bits; with size, every term by its absolute value (and M)."""
    pos = (lambda t: t.abs()) if size else (lambda t: t)
    n, c, l = d["u"].shape
    G, S = d["groups"], d["A"].shape[1]
    cg = c // G
    m = torch.full((n,), l, device=d["u"].device) if d["lengths"] is None else d["lengths"].clamp(0, l).long()
    on = torch.arange(l, device=m.device)[None] < m[:, None]
    cut = lambda t: torch.where(on[:, None], t.double(), 0.0)  # noqa: E731
    u, raw = cut(d["u"]), cut(d["delta"])
    if d["delta_bias"] is not None:
        raw = raw + d["delta_bias"].double()[:, None]
    step = torch.where(on[:, None], torch.logaddexp(raw, torch.zeros_like(raw)) if d["softplus"] else raw, 0.0)
    u = pos(u)
    Bm, Cm = (pos(cut(d[k].reshape(n, -1, l))).view(n, G, S, l) for k in "BC")
    A = d["A"].double()
    skip = torch.zeros(c, device=u.device, dtype=torch.float64) if d["D"] is None else pos(d["D"].double())
    wide = lambda t: t.repeat_interleave(cg, 1)  # noqa: E731  [N, G, S] -> [N, C, S]
    h = torch.zeros((n, c, S), dtype=torch.float64, device=u.device)
    if d["state"] is not None:
        h = pos(d["state"].double())
    hs, ys, E, M = [h], [], 2 * h, 1.0
    for t in range(l):
        a, b = torch.exp(step[:, :, t, None] * A), pos(step[:, :, t, None]) * wide(Bm[..., t]) * u[:, :, t, None]
        if size:
            E = a * (E + (1 + (step[:, :, t, None] * A).abs()) * h) + 2 * b
        h = a * h + b
        hs.append(h)
        ys.append((wide(Cm[..., t]) * h).sum(2))
        if size:
            M = max(M, float((E / h.clamp(min=1e-300))[h > 0].max()) if bool((h > 0).any()) else 1.0)
    pre = torch.stack(ys, 2) + skip[:, None] * u
    gate = dgate = 1.0
    if d["z"] is not None:
        z = cut(d["z"])
        s = torch.sigmoid(z)
        # silu' = s (1 + z (1 - s)) vanishes at z = -1.28: an error e of s, relative, moves it by e s |z| s there, so that its
        # terms' size is s (1 + |z| (1 - s) + |z| s) = s (1 + |z|)
        gate, dgate = pos(z * s), s * (1 + z.abs()) if size else s * (1 + z * (1 - s))
    got = {"y": torch.where(on[:, None], pre * gate, 0.0), "state": h, "M": M}
    if dy is None:
        return got
    dout = pos(cut(dy))
    dz = dout * pre * dgate
    g = dout * gate
    w = torch.zeros_like(h) if dstate_out is None else pos(dstate_out.double())
    du, dd = skip[:, None] * g, torch.zeros_like(u)
    dA, dB, dC = torch.zeros_like(A), torch.zeros((n, G, S, l), dtype=u.dtype, device=u.device), torch.zeros((n, G, S, l), dtype=u.dtype, device=u.device)
    share = lambda t: t.view(n, G, cg, S).sum(2)  # noqa: E731
    for t in range(l - 1, -1, -1):
        s = step[:, :, t, None]
        a, gt = torch.exp(s * A), wide(Cm[..., t]) * g[:, :, t, None] + w
        dC[..., t] = share(g[:, :, t, None] * hs[t + 1])
        dB[..., t] = share(gt * pos(s) * u[:, :, t, None])
        q = gt * a * hs[t]
        sb = (gt * wide(Bm[..., t])).sum(2)
        du[:, :, t] += pos(step[:, :, t]) * sb
        dd[:, :, t] = u[:, :, t] * sb + (q * pos(A)).sum(2)
        dA += (q * pos(s)).sum(0)
        w = a * gt
    if d["softplus"]:
        dd = dd * torch.sigmoid(raw)
    keep = lambda t: torch.where(on[:, None], t, 0.0)  # noqa: E731
    dd = keep(dd)
    got.update(du=keep(du), ddelta=dd, dA=dA, dB=torch.where(on[:, None, None], dB, 0.0), dC=torch.where(on[:, None, None], dC, 0.0),
               dD=(g * u).sum((0, 2)), ddelta_bias=dd.sum((0, 2)), dstate=w)
    if d["z"] is not None:
        got["dz"] = keep(dz)
    return got


def scan_inputs(shape, dtype, dev, seed, gated=True, skip=True, biased=True, softplus=True, carried=True, ragged=False):
    n, c, l, S, G = shape
    gen = torch.Generator().manual_seed(seed)
    t = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = {"groups": G, "softplus": softplus, "lengths": None}
    d["u"], d["B"], d["C"] = t(n, c, l).to(dtype), t(n, G * S, l).to(dtype), t(n, G * S, l).to(dtype)
    d["delta"] = (t(n, c, l) - 2 if softplus else 0.3 * torch.rand(n, c, l, generator=gen)).to(dtype)
    d["A"] = -0.2 - 3 * torch.rand(c, S, generator=gen)
    d["z"] = t(n, c, l).to(dtype) if gated else None
    d["D"] = t(c) if skip else None
    d["delta_bias"] = 0.3 * t(c) if biased and softplus else None
    d["state"] = t(n, c, S) if carried else None
    if ragged:
        d["lengths"] = torch.tensor([(l - (i * (l + 3)) // max(1, n - 1)) if n > 1 else l // 2 for i in range(n)], dtype=torch.int32)
    return {k: v.to(dev) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def forward(d, y, **kw):
    gc.gconv_scan_fwd(d["u"], d["delta"], d["A"], d["B"], d["C"], y, D=d["D"], z=d["z"], delta_bias=d["delta_bias"],
                      softplus=d["softplus"], groups=d["groups"], state=d["state"], lengths=d["lengths"], **kw)


def backward(d, dy, saved, new, dtype, **kw):
    n, c, l = d["u"].shape
    o = {k: new(d["u"].shape, dtype) for k in ("du", "ddelta")}
    o["dB"], o["dC"] = new(d["B"].shape, dtype), new(d["B"].shape, dtype)
    o["dA"], o["dD"], o["ddelta_bias"] = new(d["A"].shape, F32), new((c,), F32), new((c,), F32)
    o["dz"] = new(d["u"].shape, dtype) if d["z"] is not None else None
    o["dstate"] = new((n, *d["A"].shape), F32)
    gc.gconv_scan_bwd(d["u"], d["delta"], d["A"], d["B"], d["C"], dy, saved, o["du"], o["ddelta"], o["dA"], o["dB"], o["dC"],
                      D=d["D"], z=d["z"], delta_bias=d["delta_bias"], softplus=d["softplus"], groups=d["groups"],
                      lengths=d["lengths"], dD=o["dD"], dz=o["dz"], ddelta_bias=o["ddelta_bias"], dstate=o["dstate"], **kw)
    return {k: v for k, v in o.items() if v is not None}


def kept(d, dtype):
    size = gc.gconv_scan_saved_size(d["u"].shape, d["A"].shape[1], B_.dtype_code(dtype), d["z"] is not None)
    return torch.empty(size, dtype=torch.uint8, device=d["u"].device)


# (N, C, L, states, groups): single positions, lengths on both sides of the short form, of a run and of a tile, rows that do and
# do not begin on 16 bytes, thin and wide groups, few and many states, sequences long enough for several pieces
SHAPES = [
    (1, 1, 1, 1, 1), (2, 3, 1, 16, 1), (3, 20, 8, 16, 5), (2, 6, 9, 5, 3), (1, 33, 64, 16, 1), (2, 40, 65, 16, 2),
    (1, 64, 127, 17, 1), (4, 100, 196, 16, 5), (1, 17, 1023, 16, 1), (3, 32, 200, 64, 2), (1, 5, 72, 256, 1), (2, 8, 129, 4, 8),
    (1, 130, 512, 16, 1), (1, 8, 4096, 16, 1), (2, 12, 5001, 3, 1), (5, 70, 24, 8, 1),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_scan(dev, i, dtype):
    shape = SHAPES[i]
    for j, (gated, skip, softplus, carried, ragged) in enumerate([(True, True, True, True, True), (False, False, False, False, False)]
                                                                 if i % 2 else
                                                                 [(True, False, True, False, False), (False, True, True, True, True)]):
        d = scan_inputs(shape, dtype, dev, 10 * i + j, gated, skip, skip, softplus, carried, ragged)
        n, c, l = d["u"].shape
        new = Guarded(dev)
        y, last, saved = new((n, c, l), dtype), new((n, c, shape[3]), F32), kept(d, dtype)
        forward(d, y, state_out=last, saved=saved)
        gen = torch.Generator().manual_seed(i)
        dy = torch.randn(n, c, l, generator=gen).to(dtype).to(dev)
        dlast = torch.randn(last.shape, generator=gen).to(dev) if carried else None
        got = backward(d, dy, saved, new, dtype, dstate_out=dlast)
        ref, mag = scan_ref(d, dy, dlast), scan_ref(d, dy, dlast, size=True)
        tol = 2.0 ** -20 * (2 * mag["M"] + 8)
        near("y", y, ref["y"], mag["y"], tol, dtype)
        near("state", last, ref["state"], mag["state"], tol)
        for k, v in got.items():
            r, m = ref[k].reshape(v.shape), mag[k].reshape(v.shape)
            # sums over sequences and positions go in fp32 trees: 2^9 terms one after the other at most
            more = 2.0 ** -15 if k in ("dA", "dD", "ddelta_bias") else 2.0 ** -18
            near(k, v, r, m, tol + more, v.dtype, 2 if k == "dz" else 1)
        new.check()
        # the same bits again, and without what a call does not need
        y2 = torch.empty_like(y)
        forward(d, y2)
        assert torch.equal(y, y2)
        again = backward(d, dy, saved, lambda s, t: torch.empty(s, dtype=t, device=dev), dtype, dstate_out=dlast)
        for k in got:
            assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(131, 480, 1, 16, 1), (2051, 6, 1, 5, 2), (67, 990, 1, 20, 3)])
def test_scan_one_position_of_many(dev, shape, dtype):
    """Enough sequences that a thread takes several, some of them without a position; the state in place."""
    n, c, _, S, _ = shape
    d = scan_inputs(shape, dtype, dev, n)
    d["lengths"] = torch.tensor([0 if i % 5 == 3 else 1 for i in range(n)], dtype=torch.int32, device=dev)
    ref, mag = scan_ref(d), scan_ref(d, size=True)
    new = Guarded(dev)
    y, state, saved = new((n, c, 1), dtype), new((n, c, S), F32), kept(d, dtype)
    state.copy_(d["state"])
    forward(dict(d, state=state), y, state_out=state, saved=saved)
    tol = 2.0 ** -20 * (2 * mag["M"] + 8)
    near("y", y, ref["y"], mag["y"], tol, dtype)
    near("state", state, ref["state"], mag["state"], tol)
    assert torch.equal(state[3], d["state"][3]) and bool((y[3] == 0).all())
    marks = saved.view(torch.float32)[:n * S * c].view(n, S, c) if saved.numel() % 4 == 0 else None
    if marks is not None:
        assert torch.equal(marks.transpose(1, 2), d["state"])
    new.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("l", [70, 72])
def test_scan_channels_in_turn(dev, l, dtype):
    """So many blocks of channels that a block of the gradient takes two sets of them in turn."""
    n, c, S = 33, 510, 4
    d = scan_inputs((n, c, l, S, 1), dtype, dev, l, ragged=True)
    y, last, saved = torch.empty_like(d["u"]), torch.empty_like(d["state"]), kept(d, dtype)
    forward(d, y, state_out=last, saved=saved)
    dy = torch.randn((n, c, l), generator=torch.Generator().manual_seed(l)).to(dtype).to(dev)
    new = Guarded(dev)
    got = backward(d, dy, saved, new, dtype)
    ref, mag = scan_ref(d, dy), scan_ref(d, dy, size=True)
    tol = 2.0 ** -20 * (2 * mag["M"] + 8)
    near("y", y, ref["y"], mag["y"], tol, dtype)
    for k, v in got.items():
        # dB and dC add 510 channels, at most 2^7 of them one after the other
        more = 2.0 ** -15 if k in ("dA", "dD", "ddelta_bias") else 2.0 ** -17
        near(k, v, ref[k].reshape(v.shape), mag[k].reshape(v.shape), tol + more, v.dtype, 2 if k == "dz" else 1)
    new.check()


def test_positions_without_an_axis(dev):
    """[N, C] for one position and [N, C, H, W] for a plane are the same calls as [N, C, L]."""
    d = scan_inputs((3, 10, 1, 8, 2), F32, dev, 2)
    want, got = torch.empty((3, 10, 1), device=dev), torch.empty((3, 10), device=dev)
    forward(d, want)
    forward(dict(d, **{k: d[k][..., 0] for k in ("u", "delta", "B", "C", "z")}), got)
    assert torch.equal(got, want[..., 0])
    d = scan_inputs((2, 10, 35, 8, 2), F32, dev, 2)
    want, got = torch.empty((2, 10, 35), device=dev), torch.empty((2, 10, 5, 7), device=dev)
    forward(d, want)
    e = dict(d, **{k: d[k].view(2, 10, 5, 7) for k in ("u", "delta", "z")}, **{k: d[k].view(2, 2, 8, 5, 7) for k in "BC"})
    forward(e, got)
    assert torch.equal(got.view(2, 10, 35), want)
    x, w = torch.randn((3, 10), device=dev), torch.randn((10, 4), device=dev)
    state = torch.randn((3, 10, 3), device=dev)
    y, z = torch.empty((3, 10), device=dev), torch.empty((3, 10, 1), device=dev)
    gc.gconv_causal_fwd(x, w, None, y, state=state)
    gc.gconv_causal_fwd(x[..., None], w, None, z, state=state)
    assert torch.equal(y, z[..., 0])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_slices_in_place(dev, dtype):
    """Inputs and gradients as channel slices of larger tensors, at offsets on and off 16 bytes."""
    n, c, l, S = 3, 24, 136, 16
    for extra in (8, 3):
        d = scan_inputs((n, c, l, S, 1), dtype, dev, 5)
        dense = torch.empty((n, c, l), dtype=dtype, device=dev)
        saved = kept(d, dtype)
        forward(d, dense, saved=saved)
        dy = torch.randn((n, c, l), device=dev).to(dtype)
        want = backward(d, dy, saved, lambda s, t: torch.empty(s, dtype=t, device=dev), dtype)
        big = torch.full((n, extra + 2 * c + 2 * S, l), 9.0, dtype=dtype, device=dev)
        at = {"u": slice(extra, extra + c), "z": slice(extra + c, extra + 2 * c),
              "B": slice(extra + 2 * c, extra + 2 * c + S), "C": slice(extra + 2 * c + S, extra + 2 * c + 2 * S)}
        e = dict(d)
        for k, v in at.items():
            big[:, v] = d[k]
            e[k] = big[:, v]
        out = torch.full_like(big, 9.0)
        y = out[:, at["u"]]
        forward(e, y, saved=saved)
        assert torch.equal(y, dense)
        grad = torch.full_like(big, 9.0)
        o = {"d" + k: grad[:, v] for k, v in at.items()}
        o["ddelta"] = torch.empty_like(dense)
        f = {"dA": torch.empty_like(d["A"]), "dD": torch.empty(c, device=dev), "ddelta_bias": torch.empty(c, device=dev)}
        gc.gconv_scan_bwd(e["u"], e["delta"], e["A"], e["B"], e["C"], dy, saved, o["du"], o["ddelta"], f["dA"], o["dB"], o["dC"],
                          D=e["D"], z=e["z"], delta_bias=e["delta_bias"], dz=o["dz"], dD=f["dD"], ddelta_bias=f["ddelta_bias"])
        for k, v in {**o, **f}.items():
            assert torch.equal(v, want[k]), k
        assert bool((grad[:, :extra] == 9).all()) and bool((out[:, :extra] == 9).all()) and bool((out[:, extra + c:] == 9).all())


def test_scan_against_differences(dev):
    """dA, ddelta and du against central differences of the forward pass in 64 bits."""
    d = scan_inputs((2, 6, 40, 4, 2), F32, dev, 3)
    new = lambda s, t: torch.empty(s, dtype=t, device=dev)  # noqa: E731
    y, saved = new(d["u"].shape, F32), kept(d, F32)
    forward(d, y, saved=saved)
    dy = torch.randn_like(y)
    got = backward(d, dy, saved, new, F32)
    for name, out in (("u", "du"), ("delta", "ddelta"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("state", "dstate"), ("z", "dz")):
        e = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in d.items()}
        for flat in (0, e[name].numel() // 2, e[name].numel() - 1):
            values = []
            for step in (1e-5, -1e-5):
                f = dict(e, **{name: e[name].clone()})
                f[name].view(-1)[flat] += step
                values.append(float((scan_ref(f)["y"] * dy.double()).sum()))
            slope = (values[0] - values[1]) / 2e-5
            # second derivatives times 1e-10, cancellation of 64-bit sums: far below 1e-5 of a sum of this size
            assert abs(float(got[out].reshape(-1)[flat]) - slope) < 2e-4 * (1 + abs(slope)), (name, flat)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_then_positions(dev, dtype):
    """A prompt and then single positions, states in place, against one call over all of them."""
    n, c, l, S, k = 3, 40, 100, 16, 4
    d = scan_inputs((n, c, l, S, 2), dtype, dev, 8, carried=False)
    x = torch.randn((n, c, l), device=dev).to(dtype)
    w, b = torch.randn((c, k), device=dev), torch.randn(c, device=dev)
    whole_x, whole_y = torch.empty_like(x), torch.empty_like(x)
    gc.gconv_causal_fwd(x, w, b, whole_x, act="silu")
    forward(dict(d, u=whole_x), whole_y)
    conv_state, state = torch.zeros((n, c, k - 1), dtype=dtype, device=dev), torch.zeros((n, c, S), device=dev)
    cuts = [0, 37, 38, 39, 44, 45, 60, 100]
    for lo, hi in zip(cuts, cuts[1:]):
        piece = {key: d[key][..., lo:hi].contiguous() for key in ("delta", "B", "C", "z")}
        px, py = (torch.empty((n, c, hi - lo), dtype=dtype, device=dev) for _ in range(2))
        gc.gconv_causal_fwd(x[..., lo:hi].contiguous(), w, b, px, act="silu", state=conv_state, state_out=conv_state)
        assert torch.equal(px, whole_x[..., lo:hi])
        forward(dict(d, **piece, u=px, state=state), py, state_out=state)
        ref = whole_y[..., lo:hi].double()
        # both are fp32 sums of the same terms, rounded once
        assert bool(((py.double() - ref).abs() <= (2.0 ** -7 if dtype == BF16 else 2.0 ** -12) * ref.abs() + 2.0 ** -14).all())


def test_scan_behind_the_end(dev):
    """NaN and infinities behind a sequence's length change nothing; lengths outside [0, L] count as the nearest."""
    n, c, l, S = 5, 16, 150, 16
    for dtype in (F32, BF16):
        d = scan_inputs((n, c, l, S, 1), dtype, dev, 4)
        d["lengths"] = torch.tensor([150, 77, 0, 64, 1], dtype=torch.int32, device=dev)
        dy = torch.randn((n, c, l), device=dev).to(dtype)
        new = lambda s, t: torch.full(s, 5.0, dtype=t, device=dev)  # noqa: E731
        runs = []
        for dirty in (False, True):
            e = dict(d, **{k: d[k].clone() for k in ("u", "delta", "B", "C", "z")})
            g = dy.clone()
            if dirty:
                for i, m in enumerate([150, 77, 0, 64, 1]):
                    for j, k in enumerate(("u", "delta", "B", "C", "z")):
                        e[k][i, :, m:] = (float("nan"), float("inf"), float("-inf"))[j % 3]
                    g[i, :, m:] = float("nan")
                e["lengths"] = torch.tensor([1000, 77, -3, 64, 1], dtype=torch.int32, device=dev)
            y, last, saved = new((n, c, l), dtype), new((n, c, S), F32), kept(d, dtype)
            forward(e, y, state_out=last, saved=saved)
            runs.append({"y": y, "last": last, **backward(e, g, saved, new, dtype)})
        for k in runs[0]:
            assert torch.equal(runs[0][k], runs[1][k]), k
        assert torch.equal(runs[0]["last"][2], d["state"][2])
        assert bool((runs[0]["y"][2] == 0).all()) and bool((runs[0]["y"][1, :, 77:] == 0).all())
        assert bool((runs[0]["dB"][3, :, 64:] == 0).all()) and bool((runs[0]["du"][4, :, 1:] == 0).all())


def test_scan_special_values(dev):
    """Steps of zero, decays of zero and of minus infinity, steps beyond the exponential's range."""
    d = scan_inputs((1, 8, 80, 16, 1), F32, dev, 6, gated=False, skip=False, softplus=False, carried=True)
    d["delta"][0, 0] = 0.0
    d["A"][1] = 0.0
    d["delta"][0, 2] = 500.0
    y, last = torch.empty_like(d["u"]), torch.empty_like(d["state"])
    forward(d, y, state_out=last)
    ref, mag = scan_ref(d), scan_ref(d, size=True)
    near("y", y, ref["y"], mag["y"], 2.0 ** -20 * (2 * mag["M"] + 8))
    assert torch.equal(last[0, 0], d["state"][0, 0])
    d["A"][3] = float("-inf")
    d["u"][0, 4, 50] = float("inf")
    d["delta"][0, 5, 10] = float("nan")
    forward(d, y, state_out=last)
    alone = (d["delta"][0, 3] * d["u"][0, 3])[None] * d["B"][0]
    near("A = -inf", last[0, 3], alone[:, -1].double(), alone[:, -1].abs().double(), 2.0 ** -20)
    assert bool(torch.isfinite(y[0, 4, :50]).all()) and not bool(torch.isfinite(y[0, 4, 50:]).any())
    assert bool(torch.isfinite(y[0, 5, :10]).all()) and bool(torch.isnan(y[0, 5, 10:]).all())
    assert bool(torch.isfinite(y[0, 6:]).all())


# ---- the causal convolution ------------------------------------------------------


def causal_ref(x, w, b, act, state, lengths, dy=None, dstate_out=None, size=False):
    pos = (lambda t: t.abs()) if size else (lambda t: t)
    n, c, l = x.shape
    k = w.shape[1]
    out = {key: torch.zeros((n, c, l), dtype=torch.float64, device=x.device) for key in ("y", "dx", "v")}
    last, first = (torch.zeros((n, c, k - 1), dtype=torch.float64, device=x.device) for _ in range(2))
    dw, db = torch.zeros((c, k), dtype=torch.float64, device=x.device), torch.zeros(c, dtype=torch.float64, device=x.device)
    wd = w.double()
    for i in range(n):
        m = l if lengths is None else int(lengths[i].clamp(0, l))
        head = torch.zeros((c, k - 1), dtype=torch.float64, device=x.device) if state is None else state[i].double()
        line = torch.cat([head, x[i, :, :m].double()], 1)
        last[i] = line[:, m:]
        taps = torch.stack([line[:, j:j + m] for j in range(k)], 2)
        v = (taps * wd[:, None]).sum(2) + (0 if b is None else b.double()[:, None])
        big = (taps.abs() * wd.abs()[:, None]).sum(2) + (0 if b is None else b.double().abs()[:, None])
        s = torch.sigmoid(v)
        out["v"][i, :, :m] = v
        out["y"][i, :, :m] = (big * (s + v.abs() * s * (1 - s)) if act == "silu" else big) if size else (v * s if act == "silu" else v)
        if dy is None:
            continue
        dv = pos(dy[i, :, :m].double())
        if act == "silu":
            # |act''| < 1/2: what an error of v, relative to its terms, does to act'(v)
            dv = dv * ((s * (1 + v * (1 - s))).abs() + 0.5 * big if size else s * (1 + v * (1 - s)))
        dl = torch.zeros_like(line)
        for j in range(k):
            dl[:, j:j + m] += pos(wd[:, j, None]) * dv
        if dstate_out is not None:
            dl[:, m:] += pos(dstate_out[i].double())
        first[i], out["dx"][i, :, :m] = dl[:, :k - 1], dl[:, k - 1:]
        dw += (dv[:, :, None] * pos(taps)).sum(1)
        db += dv.sum(1)
    return dict(out, state=last, dstate=first, dw=dw, db=db)


CAUSAL = [(1, 1, 1), (2, 5, 2), (3, 8, 4), (2, 7, 5), (4, 12, 7), (2, 16, 8), (1, 33, 63), (3, 9, 64), (2, 6, 1023), (1, 4, 2048), (1, 3, 4099),
          (70, 3, 9), (2, 300, 16)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("taps", range(1, 9))
@pytest.mark.parametrize("shape", CAUSAL)
def test_causal(dev, shape, taps, dtype):
    n, c, l = shape
    gen = torch.Generator().manual_seed(l + taps)
    t = lambda *s: torch.randn(*s, generator=gen).to(dev)  # noqa: E731
    for full in (True, False):
        x, dy = t(n, c, l).to(dtype), t(n, c, l).to(dtype)
        w, b = t(c, taps), t(c) if full else None
        state = t(n, c, taps - 1).to(dtype) if full else None
        more = t(n, c, taps - 1).to(dtype) if full else None
        lengths = torch.tensor([max(0, l - 3 * i) if i % 3 else l for i in range(n)], dtype=torch.int32, device=dev) if full else None
        act = "silu" if full else "none"
        new = Guarded(dev)
        y, last = new((n, c, l), dtype), new((n, c, taps - 1), dtype)
        dx, dw, db, first = new((n, c, l), dtype), new((c, taps), F32), new((c,), F32), new((n, c, taps - 1), dtype)
        gc.gconv_causal_fwd(x, w, b, y, act=act, state=state, state_out=last, lengths=lengths)
        gc.gconv_causal_bwd(x, w, b, dy, dx, dw, db, act=act, state=state, lengths=lengths, dstate_out=more, dstate=first)
        ref = causal_ref(x, w, b, act, state, lengths, dy, more)
        mag = causal_ref(x, w, b, act, state, lengths, dy, more, size=True)
        tol = 2.0 ** -20 + 2.0 ** -22 * float(ref["v"].abs().max())
        near("y", y, ref["y"], mag["y"], tol, dtype)
        assert torch.equal(last.double(), ref["state"])
        near("dx", dx, ref["dx"], mag["dx"], tol, dtype)
        near("dstate", first, ref["dstate"], mag["dstate"], tol, dtype)
        near("dw", dw, ref["dw"], mag["dw"], tol + 2.0 ** -15)
        near("db", db, ref["db"], mag["db"], tol + 2.0 ** -15)
        new.check()
        again = torch.empty_like(dw)
        gc.gconv_causal_bwd(x, w, b, dy, dx, again, act=act, state=state, lengths=lengths, dstate_out=more)
        assert torch.equal(again, dw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("l", [65, 64])
def test_causal_slices_and_planes(dev, l, dtype):
    """Channel slices whose rows begin at the same or at another place of 16 bytes, planes [H, W], and the weights as
    the depthwise convolution has them, whose result it is."""
    n, c, k = 3, 10, 4
    big = torch.randn((n, 2 * c + 1, l), device=dev).to(dtype)
    w = torch.randn((c, 1, 1, k), device=dev)
    want = torch.empty((n, c, l), dtype=dtype, device=dev)
    for lo in (0, c, c + 1):
        x = big[:, lo:lo + c]
        gc.gconv_causal_fwd(x.contiguous(), w, None, want)
        out = torch.full_like(big, 3.0)
        gc.gconv_causal_fwd(x, w, None, out[:, 1:1 + c])
        assert torch.equal(out[:, 1:1 + c], want)
        assert bool((out[:, 0] == 3).all()) and bool((out[:, 1 + c:] == 3).all())
        dx, dw = torch.empty_like(want), torch.empty_like(w)
        gc.gconv_causal_bwd(x.contiguous(), w, None, want, dx, dw, act="silu")
        grad, dw2 = torch.full_like(big, 3.0), torch.empty_like(w)
        gc.gconv_causal_bwd(x, w, None, want, grad[:, 1:1 + c], dw2, act="silu")
        assert torch.equal(grad[:, 1:1 + c], dx) and bool((grad[:, 1 + c:] == 3).all())
        near("dw", dw2, dw.double(), dw.double().abs() + 1, 2.0 ** -15)
    x = torch.randn((2, 6, 5, 13), device=dev).to(dtype)
    w, y = torch.randn((6, 1, 1, k), device=dev), torch.empty_like(x)
    gc.gconv_causal_fwd(x, w, None, y)
    line, same = x.reshape(2, 6, 1, 65), torch.empty((2, 6, 1, 65), device=dev)
    if dtype == F32:
        gc.gconv_fwd(line, w, None, same, padding=(0, 0, k - 1, 0), groups=6)
        near("depthwise", y.reshape(same.shape), same.double(), same.double().abs() + 1, 2.0 ** -20)


def test_empty_batches(dev):
    """No sequences: nothing runs, and the parameters' gradients are zero."""
    e = lambda *s: torch.empty(s, device=dev)  # noqa: E731
    w, b, dw, db = torch.randn((6, 4), device=dev), e(6), torch.full((6, 4), 5.0, device=dev), torch.full((6,), 5.0, device=dev)
    gc.gconv_causal_fwd(e(0, 6, 9), w, b, e(0, 6, 9), state=e(0, 6, 3), state_out=e(0, 6, 3))
    gc.gconv_causal_bwd(e(0, 6, 9), w, b, e(0, 6, 9), e(0, 6, 9), dw, db)
    assert not bool(dw.any()) and not bool(db.any())
    for l in (1, 80):
        d = scan_inputs((0, 6, l, 8, 2), F32, dev, 1)
        saved = kept(d, F32)
        forward(d, e(0, 6, l), saved=saved)
        got = backward(d, e(0, 6, l), saved, lambda s, t: torch.full(s, 5.0, dtype=t, device=dev), F32)
        assert not any(bool(got[k].any()) for k in ("dA", "dD", "ddelta_bias"))
    gc.gconv_dropout_fwd(e(0), e(0), torch.zeros(2, dtype=torch.int64, device=dev), 0.5)


def test_tensors_elsewhere_are_refused(dev):
    """A tensor of the host among the device's, for each argument."""
    d = scan_inputs((2, 6, 20, 8, 1), F32, dev, 1)
    y = torch.empty_like(d["u"])
    for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias", "state"):
        with pytest.raises(ValueError):
            forward(dict(d, **{k: d[k].cpu()}), y)
    with pytest.raises(ValueError):
        forward(d, y.cpu())
    with pytest.raises(ValueError):
        forward(dict(d, lengths=torch.tensor([1, 2], dtype=torch.int32)), y)
    with pytest.raises(ValueError):
        forward(dict(d, lengths=torch.tensor([1, 2], device=dev)), y)
    with pytest.raises(ValueError):
        forward(d, y, saved=torch.empty(8, device=dev))
    w = torch.randn((6, 4), device=dev)
    for args in ((d["u"].cpu(), w, None, y), (d["u"], w.cpu(), None, y), (d["u"], w, None, y.cpu()), (d["u"], w.bfloat16(), None, y),
                 (d["u"], w, torch.zeros(5, device=dev), y), (d["u"].transpose(1, 2), w, None, y), (d["u"][:1].expand(2, 6, 20), w, None, y)):
        with pytest.raises(ValueError):
            gc.gconv_causal_fwd(*args)
    with pytest.raises(ValueError):
        gc.gconv_dropout_fwd(y, y, torch.zeros(2, dtype=torch.int64), 0.5)


def test_beyond_32_bits(dev):
    """Tensors of more than 2^31 elements: the last channels of the last sequence against a call on them alone."""
    n, c, l, S = 2, 17000, 65535, 4
    if torch.cuda.get_device_properties(dev).total_memory < 60e9:
        pytest.skip("needs 40 GB")
    gen = torch.Generator(device=dev).manual_seed(3)
    x = torch.empty((n, c, l), dtype=BF16, device=dev).normal_(generator=gen)
    delta = torch.empty_like(x).normal_(generator=gen)
    y = torch.empty_like(x)
    w, b = torch.randn((c, 4), device=dev), torch.randn(c, device=dev)
    last = lambda t: t[n - 1:, c - 3:].contiguous()  # noqa: E731
    want = torch.empty((1, 3, l), dtype=BF16, device=dev)
    gc.gconv_causal_fwd(x, w, b, y, act="silu")
    gc.gconv_causal_fwd(last(x), w[c - 3:].contiguous(), b[c - 3:].contiguous(), want, act="silu")
    assert torch.equal(last(y), want)
    B, C = (torch.randn((n, S, l), device=dev).to(BF16) for _ in range(2))
    A, D = -0.2 - torch.rand((c, S), device=dev), torch.randn(c, device=dev)
    gc.gconv_scan_fwd(x, delta, A, B, C, y, D=D)
    gc.gconv_scan_fwd(last(x), last(delta), A[c - 3:].contiguous(), B[1:].contiguous(), C[1:].contiguous(), want, D=D[c - 3:].contiguous())
    # the sequences are cut in other pieces: fp32 sums of some tens of terms that matter, then bf16
    got = last(y).double()
    assert bool(((got - want.double()).abs() <= 2.0 ** -7 * want.double().abs() + 2.0 ** -12).all())


# ---- together, captured, on another stream ------------------------------------------


def test_a_mixing_block(dev):
    """1x1 convolution -> causal convolution -> scan gated by the other half -> 1x1 convolution -> dropout onto the
    residual, forward and backward in fp32, against autograd in 64 bits: every stage's error is at most 2^-14 of its terms."""
    n, c, e, l, S, p = 2, 16, 32, 70, 8, 0.25
    gen = torch.Generator().manual_seed(1)
    t = lambda *s: torch.randn(*s, generator=gen).to(dev)  # noqa: E731
    x, w_in, w_out = t(n, c, 1, l), t(2 * e, c, 1, 1) * c ** -0.5, t(c, e, 1, 1) * e ** -0.5
    wx = t(e + 2 * S, e, 1, 1) * e ** -0.5
    w, b, A, D, bias = 0.5 * t(e, 4), 0.1 * t(e), -0.2 - 2 * torch.rand(e, S, generator=gen).to(dev), t(e), t(e) - 2
    rng, dout = torch.tensor([11, 3], device=dev), t(n, c, 1, l)
    new = lambda *s: torch.empty(s, device=dev)  # noqa: E731
    xz, v, proj, y, h, out = new(n, 2 * e, 1, l), new(n, e, 1, l), new(n, e + 2 * S, 1, l), new(n, e, 1, l), new(n, c, 1, l), new(n, c, 1, l)
    saved = torch.empty(gc.gconv_scan_saved_size((n, e, l), S, gc.GCONV_F32, True), dtype=torch.uint8, device=dev)
    gc.gconv_fwd(x, w_in, None, xz)
    gc.gconv_causal_fwd(xz[:, :e], w, b, v, act="silu")
    gc.gconv_fwd(v, wx, None, proj)
    scan = (v, proj[:, :e], A, proj[:, e:e + S], proj[:, e + S:])
    gc.gconv_scan_fwd(*scan, y, D=D, z=xz[:, e:], delta_bias=bias, saved=saved)
    gc.gconv_fwd(y, w_out, None, h)
    gc.gconv_dropout_fwd(h, out, rng, p, res=x)
    # backward
    dh, dy, dxz, dproj, dv, dv2, dx = new(n, c, 1, l), new(n, e, 1, l), new(n, 2 * e, 1, l), new(n, e + 2 * S, 1, l), new(n, e, 1, l), new(n, e, 1, l), new(n, c, 1, l)
    dw_out, dw_in, dwx, dw, db, dA, dD, dbias = (torch.empty_like(q) for q in (w_out, w_in, wx, w, b, A, D, bias))
    gc.gconv_dropout_bwd(dout, dh, rng, p)
    gc.gconv_bwd_data(dh, w_out, dy)
    gc.gconv_bwd_weight(y, dh, dw_out)
    gc.gconv_scan_bwd(*scan, dy, saved, dv, dproj[:, :e], dA, dproj[:, e:e + S], dproj[:, e + S:], D=D, z=xz[:, e:], delta_bias=bias,
                      dD=dD, dz=dxz[:, e:], ddelta_bias=dbias)
    gc.gconv_bwd_data(dproj, wx, dv2)
    gc.gconv_bwd_weight(v, dproj, dwx)
    gc.gconv_causal_bwd(xz[:, :e], w, b, dv + dv2, dxz[:, :e], dw, db, act="silu")
    gc.gconv_bwd_data(dxz, w_in, dx)
    gc.gconv_bwd_weight(x, dxz, dw_in)
    dx += dout
    # in 64 bits
    leaves = {k: q.double().requires_grad_() for k, q in dict(x=x, w_in=w_in, w_out=w_out, wx=wx, w=w, b=b, A=A, D=D, bias=bias).items()}
    q = leaves
    mask = gc.gconv_dropout_fwd(torch.ones_like(x), new(n, c, 1, l), rng, p).double()
    r = q["x"][:, :, 0]
    both = torch.einsum("oc,ncl->nol", q["w_in"][:, :, 0, 0], r)
    pad = torch.nn.functional.pad(both[:, :e], (3, 0))
    u = sum(q["w"][:, j, None] * pad[:, :, j:j + l] for j in range(4)) + q["b"][:, None]
    u = u * torch.sigmoid(u)
    pr = torch.einsum("oc,ncl->nol", q["wx"][:, :, 0, 0], u)
    step = torch.nn.functional.softplus(pr[:, :e] + q["bias"][:, None])
    state, ys = torch.zeros((n, e, S), dtype=torch.float64, device=dev), []
    for i in range(l):
        state = torch.exp(step[:, :, i, None] * q["A"]) * state + (step[:, :, i] * u[:, :, i])[..., None] * pr[:, None, e:e + S, i]
        ys.append((state * pr[:, None, e + S:, i]).sum(2))
    s = (torch.stack(ys, 2) + q["D"][:, None] * u) * torch.nn.functional.silu(both[:, e:])
    o = (torch.einsum("oc,ncl->nol", q["w_out"][:, :, 0, 0], s) * mask[:, :, 0] + r)
    got = dict(x=dx, w_in=dw_in, w_out=dw_out, wx=dwx, w=dw, b=db, A=dA, D=dD, bias=dbias)
    near("out", out[:, :, 0], o.detach(), o.detach().abs() + o.detach().std(), 2.0 ** -14)
    for k, g in zip(leaves, torch.autograd.grad(o, list(leaves.values()), dout[:, :, 0].double())):
        near("d" + k, got[k], g, g.abs() + g.std(), 2.0 ** -13)


def test_captured_and_streams(dev):
    """Captured forward and backward calls replayed on new values, and calls on a side stream, give the bits of plain calls."""
    d = scan_inputs((2, 48, 300, 16, 1), BF16, dev, 2)
    w, b = torch.randn((48, 4), device=dev), torch.randn(48, device=dev)
    dy = torch.randn((2, 48, 300), device=dev).to(BF16)
    new = lambda s, t: torch.empty(s, dtype=t, device=dev)  # noqa: E731

    def step():
        v, y, saved = torch.empty_like(d["u"]), torch.empty_like(d["u"]), kept(d, BF16)
        gc.gconv_causal_fwd(d["u"], w, b, v, act="silu")
        e = dict(d, u=v)
        forward(e, y, saved=saved)
        o = backward(e, dy, saved, new, BF16)
        dx, dw = torch.empty_like(v), torch.empty_like(w)
        gc.gconv_causal_bwd(d["u"], w, b, o["du"], dx, dw, act="silu")
        return [y, dx, dw, *o.values()]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for scale in (1.0, 0.5):
        d["u"].mul_(scale)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(step(), held))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_zeros_behind_a_length_whatever_the_weights_are(dev, dtype, act):
    x, w = torch.randn(2, 3, 512, device=dev).to(dtype), torch.randn(3, 4, device=dev)
    w[1, 0], w[2, 3] = float("inf"), float("nan")
    lengths = torch.tensor([100, 0], dtype=torch.int32, device=dev)
    y, dx, dw = torch.full_like(x, 7), torch.full_like(x, 7), torch.empty_like(w)
    gc.gconv_causal_fwd(x, w, None, y, act=act, lengths=lengths)
    gc.gconv_causal_bwd(x, w, None, x, dx, dw, act=act, lengths=lengths)
    for out in (y, dx):
        assert (out[0, :, 100:] == 0).all() and (out[1] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("l", [6, 255, 512, 4096])
def test_scan_zeros_behind_a_length_whatever_the_parameters_are(dev, dtype, l):
    n, c, S = 2, 10, 16
    x, bc = torch.randn(n, c, l, device=dev).to(dtype), torch.randn(n, S, l, device=dev).to(dtype)
    A, D, bias = -torch.rand(c, S, device=dev), torch.randn(c, device=dev), torch.randn(c, device=dev)
    A[1, 0], D[2], bias[3] = float("nan"), float("inf"), float("nan")
    state = torch.full((n, c, S), float("inf"), device=dev)
    state[0] = 1
    half = l // 2
    lengths = torch.tensor([half, 0], dtype=torch.int32, device=dev)
    new = lambda like: torch.full_like(like, 7)  # noqa: E731
    y, du, dd, dz, dB, dC, dA, dstate = new(x), new(x), new(x), new(x), new(bc), new(bc), new(A), new(state)
    saved = torch.empty(gc.gconv_scan_saved_size((n, c, l), S, 1 if dtype is BF16 else 0, gated=True), dtype=torch.uint8, device=dev)
    out = torch.empty_like(state)
    gc.gconv_scan_fwd(x, x, A, bc, bc, y, D=D, z=x, delta_bias=bias, state=state, state_out=out, lengths=lengths, saved=saved)
    gc.gconv_scan_bwd(x, x, A, bc, bc, x, saved, du, dd, dA, dB, dC, D=D, z=x, delta_bias=bias, lengths=lengths, dz=dz,
                      dstate_out=state, dstate=dstate)
    for o in (y, du, dd, dz, dB, dC):
        assert (o[0, :, half:] == 0).all() and (o[1] == 0).all()
    assert (out[1] == float("inf")).all() and (dstate[1] == float("inf")).all()
    assert torch.isfinite(dA[4:]).all() and torch.isfinite(y[0, 4:]).all()
