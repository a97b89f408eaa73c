"""Gradients of the causal convolution near the ends of its sequences, with weights that are infinite or NaN: a result that is not
there takes no part in dx or dstate."""
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from test_sequence import BF16, F32, Guarded, causal_ref, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def same(name, got, ref, mag, dtype):
    """Equal where ref is infinite or NaN; elsewhere within 8 products' roundings (2^-20 of their sum) and half a unit of dtype."""
    g = got.double()
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), name
    inf, fine = torch.isinf(ref), torch.isfinite(ref)
    assert torch.equal(g[inf], ref[inf]), name
    bound = 2.0 ** -20 * mag[fine] + (2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * ref[fine].abs() + 1e-30
    assert bool(((g[fine] - ref[fine]).abs() <= bound).all()), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("taps", [1, 2, 4, 5, 8])
@pytest.mark.parametrize("l", [1, 3, 16, 23, 64, 257, 520])
def test_weights_of_results_that_are_not_there(dev, l, taps, dtype):  # noqa: F811
    ends = sorted({l, 0, *(min(l, m) for m in (1, 2, taps - 1, taps, 8, 9, l // 2, l - 1))})
    n, c = len(ends), 2 * taps + 1
    gen = torch.Generator().manual_seed(l + taps)
    t = lambda *s: torch.randn(*s, generator=gen).to(dev)  # noqa: E731
    x, dy = t(n, c, l).to(dtype), t(n, c, l).to(dtype)
    w = t(c, taps)
    for k in range(taps):                   # one tap of a channel, the last channel none
        w[k, k], w[taps + k, k] = float("inf"), float("nan")
    state, more = t(n, c, taps - 1).to(dtype), t(n, c, taps - 1).to(dtype)
    lengths = torch.tensor(ends, dtype=torch.int32, device=dev)
    for size in (lengths, None):
        new = Guarded(dev)
        dx, dw, first = new((n, c, l), dtype), new((c, taps), F32), new((n, c, taps - 1), dtype)
        gc.gconv_causal_bwd(x, w, None, dy, dx, dw, state=state, lengths=size, dstate_out=more, dstate=first)
        ref = causal_ref(x, w, None, "none", state, size, dy, more)
        mag = causal_ref(x, w, None, "none", state, size, dy, more, size=True)
        same("dx", dx, ref["dx"], mag["dx"], dtype)
        same("dstate", first, ref["dstate"], mag["dstate"], dtype)
        new.check()
    # rows of dy that begin at another place of 16 bytes than those of x, so that no access is 16 bytes
    wide = torch.full((n, c + 1, l + 1), 3.0, dtype=dtype, device=dev).view(n, -1)[:, 1:1 + c * l].unflatten(1, (c, l))
    wide.copy_(dy)
    other, last = torch.empty_like(dx), torch.empty_like(first)
    gc.gconv_causal_bwd(x, w, None, wide, other, dw, state=state, lengths=lengths, dstate_out=more, dstate=last)
    gc.gconv_causal_bwd(x, w, None, dy, dx, dw, state=state, lengths=lengths, dstate_out=more, dstate=first)
    for p, q in ((other, dx), (last, first)):
        assert torch.equal(torch.isnan(p), torch.isnan(q)) and torch.equal(torch.nan_to_num(p), torch.nan_to_num(q))
    # of a sequence without positions the state goes on as it is, and so does its gradient, through silu too
    i = ends.index(0)
    for act in ("none", "silu"):
        gc.gconv_causal_bwd(x, w, None, dy, dx, dw, act=act, state=state, lengths=lengths, dstate_out=more, dstate=first)
        assert torch.equal(first[i], more[i])
        gc.gconv_causal_bwd(x, w, None, dy, dx, dw, act=act, state=state, lengths=lengths, dstate=first)
        assert not bool(first[i].any()) and not bool(dx[i].any())
