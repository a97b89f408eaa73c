"""Calls on another stream than the current one, without a workspace of the caller's: the memory the
binding takes must stay the call's until its kernels have run.  And the block and orthogonalisation calls
captured into a CUDA graph."""
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from bwd_gconv_fwd_gb300 import binding as B

pytestmark = pytest.mark.gpu

S, G = (4, 64, 14, 14), 2


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_gconv_fwd_gb300 import build
    build.build()
    return torch.device("cuda:0")


def calls(dev):
    """name -> (workspace bytes, call(outputs, stream), outputs)"""
    gen = torch.Generator().manual_seed(1)
    t = lambda *s, dt=torch.bfloat16: torch.randn(s, generator=gen).to(dt).to(dev)  # noqa: E731
    x, h, dy, dn = (t(*S) for _ in range(4))
    w = t(64, 32, 3, 3)
    weight, g, mom = t(64, dt=torch.float32), t(150, 200, 1, 1, dt=torch.float32), t(150, 200, 1, 1, dt=torch.float32)
    small, tiny = t(64, 64, 3, 3, dt=torch.float32), t(32, 4, 3, 3, dt=torch.float32)
    f = lambda *s: torch.empty(s, device=dev)  # noqa: E731
    b = lambda: torch.empty(S, device=dev, dtype=torch.bfloat16)  # noqa: E731
    geom = gc.geometry(S, w.shape, padding=1, groups=G)
    block = gc.gconv_block_workspace_size(S, B.GCONV_BF16, G)
    orth = gc.gconv_orthogonalize_workspace_size(g.shape)
    conv = lambda p: gc.gconv_workspace_size(geom, B.GCONV_BF16, p)  # noqa: E731
    kw = dict(padding=1, groups=G)
    return {
        "norm_bwd": (block, lambda o, s: gc.gconv_norm_bwd(x, weight, dy, o[0], o[1], groups=G, stream=s), lambda: [b(), f(64)]),
        "join_bwd": (block, lambda o, s: gc.gconv_join_bwd(h, dy, o[0], weight=weight, dweight=o[1], out=x, dnext=dn, dres=o[2],
                                                           dnext_weight=o[3], groups=G, stream=s),
                     lambda: [b(), f(64), b(), f(64)]),
        "norm_fwd": (0, lambda o, s: gc.gconv_norm_fwd(x, weight, o[0], groups=G, stream=s), lambda: [b()]),
        "join_fwd": (0, lambda o, s: gc.gconv_join_fwd(x, h, o[0], gate=dy, act="silu", weight=weight, next=o[1], groups=G, stream=s),
                     lambda: [b(), b()]),
        "orthogonalize_cluster": (0, lambda o, s: gc.gconv_orthogonalize(small, o[0], stream=s), lambda: [f(*small.shape)]),
        "muon_step_block": (0, lambda o, s: gc.gconv_muon_step(tiny, tiny, tiny, w_out=o[0], m_out=o[1], groups=8, stream=s),
                            lambda: [f(*tiny.shape), f(*tiny.shape)]),
        "orthogonalize": (orth, lambda o, s: gc.gconv_orthogonalize(g, o[0], stream=s), lambda: [f(*g.shape)]),
        "muon_step": (orth, lambda o, s: gc.gconv_muon_step(g, g, mom, w_out=o[0], m_out=o[1], stream=s),
                      lambda: [f(*g.shape), f(*g.shape)]),
        "fwd": (conv(gc.PASS_FWD), lambda o, s: gc.gconv_fwd(x, w, None, o[0], stream=s, **kw), lambda: [f(*S)]),
        "bwd_data": (conv(gc.PASS_BWD_DATA), lambda o, s: gc.gconv_bwd_data(dy, w, o[0], stream=s, **kw), lambda: [f(*S)]),
        "bwd_weight": (conv(gc.PASS_BWD_WEIGHT), lambda o, s: gc.gconv_bwd_weight(x, dy, o[0], stream=s, **kw),
                       lambda: [f(*w.shape)]),
        "bwd_bias": (gc.gconv_workspace_size((4, 64, 14, 14, 64, 1, 1, 1, 0, 0, 0, 0, 1, 1), B.GCONV_BF16, gc.PASS_BWD_BIAS),
                     lambda o, s: gc.gconv_bwd_bias(dy, o[0], stream=s), lambda: [f(64)]),
        "step": (gc.gconv_step_workspace_size(geom, B.GCONV_BF16),
                 lambda o, s: gc.gconv_step(x, w, None, dy, o[0], o[1], o[2], stream=s, **kw), lambda: [f(*S), f(*S), f(*w.shape)]),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["norm_bwd", "join_bwd", "orthogonalize", "muon_step", "fwd", "bwd_data", "bwd_weight", "bwd_bias",
                                  "step"])
def test_workspace_lives_as_long_as_its_stream_needs(dev, name, raw):
    need, call, outputs = calls(dev)[name]
    assert need > 0
    want, got = outputs(), outputs()
    call(want, None)
    fill = lambda: torch.full((need,), 255, dtype=torch.uint8, device=dev)  # noqa: E731 -- NaN in fp32, fp16 and bf16
    fill()                       # what is loaded at its first launch is loaded before the other stream is held back
    torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pool = torch.empty(need, dtype=torch.uint8, device=dev)   # that stream's pool takes its memory now
        del pool
        torch.cuda._sleep(200_000_000)   # some 100 ms, so that the call's kernels run after what follows
    call(got, side.cuda_stream if raw else side)
    taken = [fill() for _ in range(8)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert all(bool((t == 255).all()) for t in taken)


@pytest.mark.parametrize("name", ["norm_fwd", "norm_bwd", "join_fwd", "join_bwd", "orthogonalize", "orthogonalize_cluster", "muon_step",
                                  "muon_step_block"])
def test_captured_calls_replay(dev, name):
    _, call, outputs = calls(dev)[name]
    want, got = outputs(), outputs()
    call(want, None)   # what is set up at a kernel's first launch is set up before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(got, None)
    for _ in range(3):
        for t in got:
            t.fill_(7.5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert gc.gconv_check_device_error() == B.GCONV_OK
