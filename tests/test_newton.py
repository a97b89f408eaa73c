"""Newton-Schulz orthogonalisation and the Muon step on the GPU against the iteration in 64 bits.

Tolerances (2-norm of the difference over the 2-norm of the result).  The iterates have 11 bits:
a rounding is off by 2^-12 of an element on average, a step multiplies what is there by up to
3.44 in the directions of small singular values and by less than one near one, and three
roundings stand in a step.  A matrix of independent normal entries whose smallest singular
value is s / sqrt(m) amplifies by about sqrt(m) / s in all, spread over m directions: 5 steps x
3 roundings x 2^-12 = 3.7e-3, taken as WELL = 4e-3.  Singular values over three decades amplify
the first rounding by 3.44^4 = 140 on an m x n matrix whose roundings share the norm 2^-12 of
the whole: 140 x 2^-12 / sqrt(8) at m = 8 or more, taken as ILL = 2.5e-2.  A bf16 result adds its
rounding, 2^-9 on average.
"""
import numpy as np
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from bwd_gconv_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)
WELL, ILL, BF16 = 4e-3, 2.5e-2, 2.0 ** -9


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_gconv_fwd_gb300 import build
    build.build()
    return torch.device("cuda:0")


def orth(g, groups, steps=5, coeffs=None, eps=1e-7):
    coeffs = [NS] * steps if coeffs is None else coeffs
    x = g.double().reshape(groups, g.shape[0] // groups, -1)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    for a, b, c in coeffs:
        gram = x @ x.mT
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.reshape(g.shape)


def off(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def normal(shape, dev, seed, dtype=torch.float32, sd=1e-3):
    return (sd * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(dtype).to(dev)


# (C_out, C_in / G, kH, kW, G): from single rows to several tiles, wide and tall, sides that are no
# multiple of any tile
SHAPES = [
    (8, 1, 3, 3, 8), (128, 4, 3, 3, 32), (5, 7, 1, 1, 1), (64, 64, 3, 3, 1), (64, 64, 1, 1, 1), (256, 48, 5, 5, 2),
    (256, 64, 1, 1, 1), (300, 5, 2, 4, 1), (129, 65, 1, 2, 1), (200, 37, 3, 3, 1), (3, 1111, 1, 2, 1), (700, 513, 1, 1, 1),
    (512, 128, 1, 1, 2), (96, 16, 3, 3, 3), (1024, 300, 1, 1, 1), (40, 2000, 1, 3, 1), (260, 130, 1, 1, 2), (1, 1, 1, 9, 1),
]


@pytest.mark.parametrize("dtype,out_dtype", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32),
                                             (torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16)])
@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalize(dev, shape, dtype, out_dtype):
    *s, G = shape
    g = normal(s, dev, 1, dtype)
    n = g.numel()
    buf = torch.full((n + 128,), 7.5, device=dev, dtype=out_dtype)
    out = buf[64:64 + n].view(s)
    gc.gconv_orthogonalize(g, out, groups=G)
    assert gc.gconv_check_device_error() == 0
    assert bool((buf[:64] == 7.5).all()) and bool((buf[64 + n:] == 7.5).all())
    assert off(out, orth(g, G)) <= WELL + (BF16 if out_dtype == torch.bfloat16 else 0.0)
    again = torch.empty_like(g, dtype=out_dtype)
    gc.gconv_orthogonalize(g, again, groups=G)
    assert torch.equal(out, again)


# (rows, cols) on a cluster of blocks whose last one has few columns of the longer side or none, where what
# the others send may land on values that a block still has to read: tall and wide, odd sides, one
# and several chunks of 64 columns a block, clusters of eight and sixteen
CLUSTERS = [(1728, 96), (1792, 96), (3712, 96), (1040, 33), (64, 1089), (64, 1025), (64, 1152), (64, 1600), (96, 1152),
            (128, 1200), (120, 4000)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", CLUSTERS)
def test_clusters_with_narrow_blocks(dev, rows, cols, dtype):
    g = normal((rows, cols, 1, 1), dev, 12, dtype)
    out, again = torch.empty_like(g, dtype=torch.float32), torch.empty_like(g, dtype=torch.float32)
    gc.gconv_orthogonalize(g, out)
    assert gc.gconv_check_device_error() == 0
    assert off(out, orth(g, 1)) <= WELL
    for _ in range(50):
        gc.gconv_orthogonalize(g, again)
        assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(32, 4, 3, 3, 8), (64, 64, 3, 3, 1), (1728, 96, 1, 1, 1), (64, 1089, 1, 1, 1), (300, 150, 1, 3, 1),
                                   (260, 130, 1, 1, 2)])
def test_in_place(dev, shape, dtype):
    *s, G = shape
    g = normal(s, dev, 17, dtype)
    want = torch.empty_like(g)
    gc.gconv_orthogonalize(g, want, groups=G)
    gc.gconv_orthogonalize(g, g, groups=G)
    assert torch.equal(g, want)


@pytest.mark.parametrize("rows,cols", [(1728, 96), (64, 1089)])
def test_muon_on_clusters_with_narrow_blocks(dev, rows, cols):
    w, grad, mom = (normal((rows, cols, 1, 1), dev, 13 + k, sd=sd) for k, sd in enumerate((0.1, 1e-3, 3e-3)))
    w2, m2 = torch.empty_like(w), torch.empty_like(w)
    gc.gconv_muon_step(w, grad, mom, w_out=w2, m_out=m2, lr=0.02, beta=0.9)
    m = 0.9 * mom.double() + grad.double()
    o = orth(grad.double() + 0.9 * m, 1)
    rate = 0.02 * max(1.0, rows / cols) ** 0.5
    assert off(m2, m) <= 1e-6
    assert float((w2.double() - w.double() + rate * o).norm()) <= WELL * rate * float(o.norm()) + 1e-6 * float(w.norm())


@pytest.mark.parametrize("m,n", [(16, 144), (64, 576), (128, 1200), (200, 200), (300, 900)])
def test_wide_spectrum(dev, m, n):
    gen = torch.Generator().manual_seed(3)
    u, _, v = torch.linalg.svd(torch.randn(m, n, generator=gen).double(), full_matrices=False)
    g = (u @ torch.diag(10.0 ** (-3 * torch.arange(m) / (m - 1))).double() @ v).float().to(dev).contiguous()
    out = torch.empty_like(g)
    gc.gconv_orthogonalize(g, out)
    assert off(out, orth(g, 1)) <= ILL


@pytest.mark.parametrize("shape", [(32, 40, 1, 1), (160, 200, 1, 1)])
def test_steps_and_coefficients(dev, shape):
    g = normal(shape, dev, 4)
    out = torch.empty_like(g)
    per_step = [(4.0, -6.0, 2.5), (3.0, -3.5, 1.3), (1.875, -1.25, 0.375)]
    gc.gconv_orthogonalize(g, out, steps=3, coeffs=per_step)
    assert off(out, orth(g, 1, coeffs=per_step)) <= WELL
    gc.gconv_orthogonalize(g, out, steps=1, coeffs=(1.5, -0.5, 0.0))
    assert off(out, orth(g, 1, 1, [(1.5, -0.5, 0.0)])) <= WELL
    with pytest.raises(ValueError):
        gc.gconv_orthogonalize(g, out, steps=3, coeffs=per_step[:2])


@pytest.mark.parametrize("s", [(12, 6, 3, 3), (260, 140, 1, 1)])
def test_zero_nan_and_scale(dev, s):
    """A zero group gives zeros, a NaN spoils its own group, sizes from 1e-15 to 1e15 do not matter."""
    g = normal((2 * s[0],) + s[1:], dev, 5)
    want = torch.empty_like(g)
    gc.gconv_orthogonalize(g, want, groups=2)
    bad = g.clone()
    bad[0] = float("nan")
    out = torch.empty_like(g)
    gc.gconv_orthogonalize(bad, out, groups=2)
    assert bool(torch.isnan(out[:s[0]]).all()) and torch.equal(out[s[0]:], want[s[0]:])
    bad = g.clone()
    bad[s[0]:] = 0
    gc.gconv_orthogonalize(bad, out, groups=2)
    assert bool((out[s[0]:] == 0).all()) and torch.equal(out[:s[0]], want[:s[0]])
    for size in (1e-12, 1e18):
        gc.gconv_orthogonalize(g * size, out, groups=2, eps=0.0)
        assert off(out, orth(g, 2)) <= WELL


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-7])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("s", [(12, 6, 3, 3), (64, 64, 3, 3), (96, 33, 1, 1), (260, 140, 1, 1), (140, 260, 1, 1)])
def test_zero_groups_for_any_eps(dev, s, dtype, eps):
    """A group of zeros gives zeros, and its weights decay only, on one block, a cluster and by products."""
    g = normal((2 * s[0],) + s[1:], dev, 15, dtype)
    want, out = torch.empty_like(g, dtype=torch.float32), torch.empty_like(g, dtype=torch.float32)
    gc.gconv_orthogonalize(g, want, groups=2, eps=eps)
    bad = g.clone()
    bad[s[0]:] = 0
    gc.gconv_orthogonalize(bad, out, groups=2, eps=eps)
    assert bool((out[s[0]:] == 0).all()) and torch.equal(out[:s[0]], want[:s[0]])
    w, mom, grad = normal(g.shape, dev, 16, sd=0.1), torch.zeros_like(want), bad.float()
    w2, m2 = torch.empty_like(w), torch.empty_like(w)
    gc.gconv_muon_step(w, grad, mom, w_out=w2, m_out=m2, groups=2, lr=0.02, weight_decay=0.1, eps=eps)
    assert float((w2[s[0]:] - (1 - 0.02 * 0.1) * w[s[0]:]).abs().max()) <= 1e-6 * float(w.abs().max())
    assert bool(torch.isfinite(w2).all())


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(64, 64, 3, 3, 1), (256, 64, 1, 1, 1), (128, 4, 3, 3, 32), (256, 48, 5, 5, 2), (300, 150, 1, 3, 1)])
def test_muon_step(dev, shape, nesterov):
    *s, G = shape
    fan = s[1] * s[2] * s[3]
    w, grad, mom = normal(s, dev, 6, sd=fan ** -0.5), normal(s, dev, 7), normal(s, dev, 8, sd=3e-3)
    lr, beta, wd = 0.02, 0.9, 0.1
    w2, m2, wb = torch.empty_like(w), torch.empty_like(w), torch.empty_like(w, dtype=torch.bfloat16)
    gc.gconv_muon_step(w, grad, mom, w_out=w2, m_out=m2, w_bf16=wb, groups=G, lr=lr, beta=beta, weight_decay=wd, nesterov=nesterov)
    m = beta * mom.double() + grad.double()
    o = orth(grad.double() + beta * m if nesterov else m, G)
    scale = max(1.0, s[0] / G / fan) ** 0.5
    ref = (1 - lr * wd) * w.double() - lr * scale * o
    assert off(m2, m) <= 1e-6
    assert float((w2.double() - ref).norm()) <= WELL * lr * scale * float(o.norm()) + 1e-6 * float(ref.norm())
    assert torch.equal(wb, w2.to(torch.bfloat16))
    gc.gconv_muon_step(w, grad, mom, groups=G, lr=lr, beta=beta, weight_decay=wd, nesterov=nesterov)   # in place
    assert torch.equal(w, w2) and torch.equal(mom, m2)


def test_other_stream_and_given_workspace(dev):
    g = normal((150, 200, 1, 1), dev, 9)
    want, got = torch.empty_like(g), torch.empty_like(g)
    gc.gconv_orthogonalize(g, want)
    need = gc.gconv_orthogonalize_workspace_size(g.shape)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    gc.gconv_orthogonalize(g, got, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(want, got)
    with pytest.raises(gc.GconvError):
        gc.gconv_orthogonalize(g, got, workspace=ws[:need - 256])


def test_refusals(dev):
    g = normal((12, 6, 3, 3), dev, 10)
    out = torch.empty_like(g)
    for bad in (lambda: gc.gconv_orthogonalize(g, out, groups=5),
                lambda: gc.gconv_orthogonalize(g, out, steps=0),
                lambda: gc.gconv_orthogonalize(g, out, steps=65),
                lambda: gc.gconv_orthogonalize(g, out, eps=-1.0),
                lambda: gc.gconv_orthogonalize(g, out, coeffs=(1.0, float("nan"), 0.0)),
                lambda: gc.gconv_orthogonalize(g, out[:6]),
                lambda: gc.gconv_orthogonalize(g.half(), out),
                lambda: gc.gconv_orthogonalize(g.permute(1, 0, 2, 3), out.permute(1, 0, 2, 3)),
                lambda: gc.gconv_orthogonalize(g.cpu(), out),
                lambda: gc.gconv_muon_step(g, g.bfloat16(), out),
                lambda: gc.gconv_muon_step(g, g, out, w_bf16=out),
                lambda: gc.gconv_muon_step(g, g, out, lr=float("inf"))):
        with pytest.raises((gc.GconvError, ValueError, TypeError)):
            bad()


@pytest.mark.parametrize("shape", [(150, 200, 1, 1), (64, 300, 1, 1), (64, 64, 1, 1)])
def test_wait_timeout_is_reported_and_recovered(dev, shape):
    """With a wait limit of zero a device-side wait that is not over at its first poll gives up (a poll
    may itself last as long as a short product): the call then reports it, else its result is right,
    and either way the next call, with the limit restored, is right."""
    g = normal(shape, dev, 11)
    out = torch.empty_like(g)
    gc.gconv_orthogonalize(g, out, steps=1)
    assert gc.gconv_check_device_error() == 0
    B.gconv_debug_set_wait_limit(0)
    try:
        gc.gconv_orthogonalize(g, out, steps=1)
        status = gc.gconv_check_device_error()
    finally:
        B.gconv_debug_set_wait_limit(-1)
    assert status == B.GCONV_ERR_TIMEOUT or (status == B.GCONV_OK and off(out, orth(g, 1, 1)) <= WELL)
    gc.gconv_orthogonalize(g, out)
    assert gc.gconv_check_device_error() == 0
    assert off(out, orth(g, 1)) <= WELL


def test_residual_block_example(dev):
    """The example's block: its output and every gradient against 64-bit autograd of the same block,
    and its training.  Eight tensors are rounded to bf16 on the longest path (2^-9 each on
    average, in root mean square adding to 0.6 %); 3 % is allowed."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "residual_block.py")
    spec = importlib.util.spec_from_file_location("residual_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    C, G, N, hw = 64, 4, 4, 12
    net = ex.Block(C, G, dev, 3)
    x, gate, dy = (normal((N, C, hw, hw), dev, 20 + k, torch.bfloat16, 1.0) for k in range(3))
    y = net.forward(x, gate)
    dx, dgate = net.backward(dy)
    v = {k: t.double().requires_grad_() for k, t in {**net.vec, "x": x, "gate": gate, **{"w_" + k: t for k, t in net.bf16.items()}}.items()}
    unit = lambda t: t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6)  # noqa: E731
    col = lambda t: t[:, None, None]  # noqa: E731
    conv = torch.nn.functional.conv2d
    h = conv(unit(v["x"]) * col(v["norm"]), v["w_mid"], padding=1, groups=G)
    s = v["x"] + col(v["scale"]) * v["gate"] * torch.sigmoid(v["gate"]) * unit(h) * col(v["weight"])
    ref = conv(unit(s) * col(v["next"]), v["w_out"])
    assert off(y, ref.detach()) <= 0.03
    got = {"x": dx, "gate": dgate, **net.dvec, **{"w_" + k: t for k, t in net.grad.items()}}
    grads = torch.autograd.grad(ref, list(v.values()), dy.double())
    for k, g in zip(v, grads):
        assert off(got[k], g) <= 0.03, k
    losses = ex.train(steps=30)
    assert losses[-1] < losses[0] and all(v == v for v in losses)
