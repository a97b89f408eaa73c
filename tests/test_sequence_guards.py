"""What the sequence calls write besides their outputs, the workspace and what is kept for the gradient, between guard words: of exactly
the sizes that are asked for, with the same results as in larger ones."""
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from test_sequence import BF16, F32, backward, dev, forward, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu
EDGE = 4096


class Bytes:
    """Buffers of bytes between guards that must come back untouched."""

    def __init__(self, dev):  # noqa: F811
        self.dev, self.bufs = dev, []

    def __call__(self, size):
        buf = torch.full((EDGE + size + EDGE,), 0x5A, dtype=torch.uint8, device=self.dev)
        self.bufs.append((buf, size))
        return buf[EDGE:EDGE + size]

    def check(self):
        for buf, size in self.bufs:
            assert bool((buf[:EDGE] == 0x5A).all()) and bool((buf[EDGE + size:] == 0x5A).all()), "write outside a buffer"


# (N, C, L, states, groups): the short form, one piece and several, one block of channels, several and sets of them, rows off 16
# bytes, more states than fit at once
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (3, 20, 8, 16, 5), (2, 3, 9, 5, 3), (1, 33, 64, 16, 1), (2, 40, 65, 16, 2), (1, 64, 127, 17, 1),
                                   (4, 100, 196, 16, 5), (3, 32, 200, 64, 2), (1, 5, 72, 256, 1), (1, 7, 4099, 3, 1), (1, 200, 4096, 16, 1),
                                   (33, 510, 70, 4, 1), (33, 511, 72, 3, 1)])
def test_scan_workspace_and_kept(dev, shape, gated, dtype):  # noqa: F811
    n, c, l, S, G = shape
    code = gc.GCONV_BF16 if dtype == BF16 else gc.GCONV_F32
    d = scan_inputs(shape, dtype, dev, sum(shape), gated=gated, ragged=True)
    dy = torch.randn((n, c, l), generator=torch.Generator().manual_seed(l)).to(dtype).to(dev)
    last = torch.randn((n, c, S), generator=torch.Generator().manual_seed(S)).to(dev)
    new = lambda s, t: torch.empty(s, dtype=t, device=dev)  # noqa: E731
    size = gc.gconv_scan_saved_size((n, c, l), S, code, gated)
    guarded, runs = Bytes(dev), []
    for take in (lambda k: torch.empty(k + 4096, dtype=torch.uint8, device=dev), guarded):
        saved = take(size)
        needs = [gc.gconv_scan_workspace_size((n, c, l), S, code, G, back) for back in (False, True)]
        work = [take(k) if k else None for k in needs]
        y, out = new((n, c, l), dtype), new((n, c, S), F32)
        forward(d, y, state_out=out, saved=saved, workspace=work[0])
        runs.append({"y": y, "out": out, **backward(d, dy, saved, new, dtype, dstate_out=last, workspace=work[1])})
        if take is guarded:
            guarded.check()
            # the last byte is asked for: one fewer is refused
            for k, w in zip((0, 1), work):
                if w is None:
                    continue
                with pytest.raises(gc.GconvError):
                    (forward(d, y, workspace=w[:-1]) if k == 0 else backward(d, dy, saved, new, dtype, workspace=w[:-1]))
            with pytest.raises(ValueError):
                forward(d, y, saved=saved[:-1])
    for k in runs[0]:
        assert torch.equal(runs[0][k], runs[1][k]), k
    guarded.check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 9, 64), (2, 6, 1023), (6, 4096, 303), (5, 9801, 41)])
def test_causal_workspace(dev, shape, dtype):  # noqa: F811
    n, c, l = shape
    code = gc.GCONV_BF16 if dtype == BF16 else gc.GCONV_F32
    gen = torch.Generator().manual_seed(l)
    x, dy = (torch.randn(shape, generator=gen).to(dtype).to(dev) for _ in range(2))
    for taps in (1, 4):
        w, b = torch.randn((c, taps), generator=gen).to(dev), torch.randn(c, generator=gen).to(dev)
        guarded, got = Bytes(dev), []
        for workspace in (None, guarded(gc.gconv_causal_workspace_size(shape, taps, code))):
            dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
            gc.gconv_causal_bwd(x, w, b, dy, dx, dw, db, act="silu", workspace=workspace)
            got.append((dx, dw, db))
        assert all(torch.equal(p, q) for p, q in zip(*got))
        guarded.check()
        with pytest.raises(gc.GconvError):
            gc.gconv_causal_bwd(x, w, b, dy, dx, dw, db, act="silu", workspace=workspace[:-1])
