"""The gradient of the scan's gate in bf16 has one rounding: the sum before the gate, which it is a product with, stays in fp32."""
import pytest
import torch

from test_sequence import BF16, Guarded, backward, dev, forward, kept, near, scan_inputs, scan_ref  # noqa: F401

pytestmark = pytest.mark.gpu


# (N, C, L, states, groups): the short form's lengths, rows on and off 16 bytes, several pieces, several blocks and sets of channels,
# more states than shared memory holds at once
@pytest.mark.parametrize("shape", [(2, 40, 1, 16, 1), (3, 20, 8, 16, 5), (2, 40, 64, 16, 2), (4, 100, 196, 16, 5), (1, 64, 127, 17, 1),
                                   (3, 32, 200, 64, 2), (1, 8, 4096, 16, 1), (2, 12, 5001, 3, 1), (33, 510, 70, 4, 1), (33, 510, 72, 4, 1)])
@pytest.mark.parametrize("skip", [True, False])
def test_dz_has_one_rounding(dev, shape, skip):  # noqa: F811
    d = scan_inputs(shape, BF16, dev, sum(shape), skip=skip, ragged=True)
    y, saved = torch.empty_like(d["u"]), kept(d, BF16)
    forward(d, y, saved=saved)
    dy = torch.randn(d["u"].shape, generator=torch.Generator().manual_seed(shape[2])).to(BF16).to(dev)
    new = Guarded(dev)
    got = backward(d, dy, saved, new, BF16)
    ref, mag = scan_ref(d, dy), scan_ref(d, dy, size=True)
    # the sum over the states within 2^-20 (2 M + 8) of its terms, the products with dy and silu' 2^-18, then half a unit of bf16
    near("dz", got["dz"], ref["dz"], mag["dz"], 2.0 ** -20 * (2 * mag["M"] + 8) + 2.0 ** -18, BF16)
    new.check()
