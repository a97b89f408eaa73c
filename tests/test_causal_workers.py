"""The causal convolution where a worker has many pieces: several rows one after the other, whole warps and parts of one, rows on and
off 16 bytes, lengths, states and their gradients."""
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from test_sequence import BF16, F32, Guarded, causal_ref, dev, near  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("taps", [1, 4, 8])
@pytest.mark.parametrize("shape", [(6, 4096, 304), (6, 4096, 303), (5, 9800, 40), (5, 9801, 41), (19, 9728, 9), (3, 20000, 65)])
def test_many_pieces_a_worker(dev, shape, taps, dtype):  # noqa: F811
    n, c, l = shape
    code = gc.GCONV_BF16 if dtype == BF16 else gc.GCONV_F32
    # the gradient's workspace is a row of sums for every worker that shares a channel: fewer of them than sequences
    splits = gc.gconv_causal_workspace_size(shape, taps, code) // (c * (taps + 1) * 4)
    assert 1 <= splits < n
    gen = torch.Generator().manual_seed(l + taps)
    t = lambda *s: torch.randn(*s, generator=gen).to(dev)  # noqa: E731
    for full in (True, False):
        x, dy = t(n, c, l).to(dtype), t(n, c, l).to(dtype)
        w, b = t(c, taps), t(c) if full else None
        state = t(n, c, taps - 1).to(dtype) if full else None
        more = t(n, c, taps - 1).to(dtype) if full else None
        lengths = torch.tensor([(l, 0, l // 2, 1, l - 1)[i % 5] for i in range(n)], dtype=torch.int32, device=dev) if full else None
        act = "silu" if full else "none"
        new = Guarded(dev)
        y, last = new((n, c, l), dtype), new((n, c, taps - 1), dtype)
        dx, dw, db, first = new((n, c, l), dtype), new((c, taps), F32), new((c,), F32), new((n, c, taps - 1), dtype)
        gc.gconv_causal_fwd(x, w, b, y, act=act, state=state, state_out=last, lengths=lengths)
        gc.gconv_causal_bwd(x, w, b, dy, dx, dw, db, act=act, state=state, lengths=lengths, dstate_out=more, dstate=first)
        ref = causal_ref(x, w, b, act, state, lengths, dy, more)
        mag = causal_ref(x, w, b, act, state, lengths, dy, more, size=True)
        # 8 products and the sigmoid 2^-20, its argument's rounding |v| 2^-22; a channel's sum has at most N L = 2^11 terms, of which
        # a lane adds at most 2^9 one after the other
        tol = 2.0 ** -20 + 2.0 ** -22 * float(ref["v"].abs().max())
        near("y", y, ref["y"], mag["y"], tol, dtype)
        assert torch.equal(last.double(), ref["state"])
        near("dx", dx, ref["dx"], mag["dx"], tol, dtype)
        near("dstate", first, ref["dstate"], mag["dstate"], tol, dtype)
        near("dw", dw, ref["dw"], mag["dw"], tol + 2.0 ** -15)
        near("db", db, ref["db"], mag["db"], tol + 2.0 ** -15)
        new.check()
        if full:                            # the state in place
            inside = state.clone()
            gc.gconv_causal_fwd(x, w, b, y, act=act, state=inside, state_out=inside, lengths=lengths)
            assert torch.equal(inside, last)
            near("y", y, ref["y"], mag["y"], tol, dtype)
