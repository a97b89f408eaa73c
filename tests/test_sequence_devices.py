"""Tensors and workspaces of another device: refused by the sequence calls before anything is kept or launched.  Without a GPU, on
stand-ins that have what the binding asks a tensor for."""
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from bwd_gconv_fwd_gb300 import binding as B


class Tensor:
    """A dense CUDA tensor by its answers only; its memory is not there."""

    is_cuda = True

    def __init__(self, *shape, dtype=torch.float32, device=1):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", device)

    def __getitem__(self, i):
        return Tensor(*self.shape[1:], dtype=self.dtype, device=self.device.index)

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize


@pytest.fixture
def current(monkeypatch):
    """Device 0 is the current one, and no call reaches the library's entry points."""
    from bwd_gconv_fwd_gb300 import build
    build.build()
    real, reached = B.lib(), []

    class Library:
        def __getattr__(self, name):
            return getattr(real, name) if name.endswith("_size") else lambda *a: reached.append(name) or 0

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0)
    monkeypatch.setattr(B, "lib", lambda: Library())
    B._causal_record.cache_clear()
    B._scan_record.cache_clear()
    return reached


def calls(device, workspace=None):
    """The sequence calls on tensors of `device`, of which all but the first need a workspace."""
    t = lambda *s, **k: Tensor(*s, device=device, **k)  # noqa: E731
    x, w, A, bc = t(2, 8, 3000), t(8, 4), t(8, 16), t(2, 16, 3000)
    saved = t(1 << 24, dtype=torch.uint8)
    kw = {} if workspace is None else {"workspace": workspace}
    return [lambda: gc.gconv_causal_fwd(x, w, None, x),
            lambda: gc.gconv_causal_bwd(x, w, None, x, x, w, **kw),
            lambda: gc.gconv_scan_fwd(x, x, A, bc, bc, x, **kw),
            lambda: gc.gconv_scan_bwd(x, x, A, bc, bc, x, saved, x, x, A, bc, bc, **kw)]


def test_tensors_of_another_device(current):
    for call in calls(1, Tensor(1 << 24, dtype=torch.uint8, device=1)):
        with pytest.raises(ValueError, match="current device"):
            call()
    # sizes are those of the current device: none may be kept for the other one
    assert B._causal_record.cache_info().currsize == 0 and B._scan_record.cache_info().currsize == 0
    assert not current


def test_workspaces_of_another_device(current):
    for call in calls(0, Tensor(1 << 24, dtype=torch.uint8, device=1))[1:]:
        with pytest.raises(ValueError, match="workspace"):
            call()
    assert not current
    for call in calls(0, Tensor(1 << 24, dtype=torch.uint8, device=0)):
        call()
    assert current == ["gconv_causal_fwd", "gconv_causal_bwd", "gconv_scan_fwd", "gconv_scan_bwd"]


def test_workspaces_of_the_matrix_calls(current):
    g = Tensor(64, 64, 3, 3, device=0)
    with pytest.raises(ValueError, match="workspace"):
        gc.gconv_orthogonalize(g, g, workspace=Tensor(1 << 24, dtype=torch.uint8, device=1))
    assert not current
