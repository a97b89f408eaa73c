"""The scan's state in place, where blocks of one piece of a sequence read it and those of another write it."""
import pytest
import torch

from test_sequence import BF16, F32, Guarded, dev, forward, scan_inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 8, 4096, 16, 1), (2, 12, 5001, 3, 1), (1, 200, 4096, 16, 1), (33, 510, 72, 4, 1), (2, 40, 65, 33, 2)])
def test_state_in_place(dev, shape, dtype):  # noqa: F811
    n, c, l, S, _ = shape
    for ragged in (False, True):
        d = scan_inputs(shape, dtype, dev, sum(shape), ragged=ragged)
        new = Guarded(dev)
        y, last, again, state = new((n, c, l), dtype), new((n, c, S), F32), new((n, c, l), dtype), new((n, c, S), F32)
        forward(d, y, state_out=last)
        state.copy_(d["state"])
        forward(dict(d, state=state), again, state_out=state)
        assert torch.equal(y, again) and torch.equal(last, state)
        new.check()
