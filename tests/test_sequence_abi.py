"""Causal convolution and selective scan entry points without a GPU: sizes and refusals, none of which reaches a launch."""
import ctypes

import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from bwd_gconv_fwd_gb300 import binding as B

BAD = ctypes.c_size_t(-1).value
OK = 1 << 20      # an aligned address that is never touched
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from bwd_gconv_fwd_gb300 import build
    build.build()
    return B.lib()


def causal(N=2, C=8, L=30, taps=4, act=0, **kw):
    return B.Causal(N, C, L, taps, act, *[kw.get(k, 0) for k in ("x_batch", "y_batch", "dy_batch", "dx_batch")])


def scan(N=2, C=8, L=30, groups=2, states=16, softplus=1, **kw):
    return B.Scan(N, C, L, groups, states, softplus, *[kw.get(k + "_batch", 0) for k in ("u", "delta", "z", "B", "C", "y", "dy", "du",
                                                                                        "ddelta", "dz", "dB", "dC")])


def causal_calls(L, r, x=OK, w=OK, bias=OK, state=OK, lengths=OK, y=OK, out=OK, dt=0):
    return [L.gconv_causal_fwd(r, dt, x, w, bias, state, lengths, y, out, None),
            L.gconv_causal_bwd(r, dt, x, w, bias, state, lengths, y, out, y, w, bias, out, OK, BIG, None)]


def scan_calls(L, r, u=OK, A=OK, Bm=OK, z=OK, D=OK, y=OK, state=OK, saved=OK, lengths=OK, dt=0, ws=OK):
    return [L.gconv_scan_fwd(r, dt, u, u, A, Bm, Bm, D, z, D, state, lengths, y, state, saved, ws, BIG, None),
            L.gconv_scan_bwd(r, dt, u, u, A, Bm, Bm, D, z, D, lengths, saved, y, state, y, y, A, Bm, Bm, D, z, D, state, ws, BIG, None)]


@pytest.mark.parametrize("r", [causal(N=-1), causal(C=0), causal(L=0), causal(taps=0), causal(taps=9), causal(act=1), causal(act=3),
                               causal(act=-1), causal(x_batch=239), causal(x_batch=-240), causal(dy_batch=1 << 41),
                               causal(N=2 ** 20, C=2 ** 20, L=2 ** 10)])
def test_invalid_causal_records(L, r):
    p = ctypes.byref(r)
    assert L.gconv_causal_workspace_size(p, 0) == BAD
    assert all(s == B.GCONV_ERR_INVALID_ARG for s in causal_calls(L, p))


@pytest.mark.parametrize("r", [scan(N=-1), scan(C=0), scan(L=0), scan(groups=0), scan(groups=3), scan(states=0), scan(states=257),
                               scan(softplus=2), scan(u_batch=239), scan(B_batch=959), scan(dC_batch=-1), scan(z_batch=1 << 41),
                               scan(N=2 ** 20, C=2 ** 20, L=2 ** 10), scan(C=2 ** 24, states=256, N=1, L=1)])
def test_invalid_scan_records(L, r):
    p = ctypes.byref(r)
    assert L.gconv_scan_saved_size(p, 0, 1) == BAD
    assert L.gconv_scan_workspace_size(p, 0, 0) == BAD and L.gconv_scan_workspace_size(p, 0, 1) == BAD
    assert all(s == B.GCONV_ERR_INVALID_ARG for s in scan_calls(L, p))


def test_null_records_and_dtypes(L):
    assert L.gconv_causal_workspace_size(None, 0) == BAD and L.gconv_scan_saved_size(None, 0, 0) == BAD
    assert all(s == B.GCONV_ERR_INVALID_ARG for s in causal_calls(L, None) + scan_calls(L, None))
    for dt in (2, -1):
        assert all(s == B.GCONV_ERR_INVALID_ARG for s in causal_calls(L, ctypes.byref(causal()), dt=dt))
        assert all(s == B.GCONV_ERR_INVALID_ARG for s in scan_calls(L, ctypes.byref(scan()), dt=dt))


def test_pointers(L):
    r = ctypes.byref(causal())
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(x=OK + 1), dict(w=OK + 2), dict(bias=OK + 2), dict(state=OK + 2),
                dict(lengths=OK + 2), dict(y=OK + 2), dict(out=OK + 2)):
        assert all(s == B.GCONV_ERR_INVALID_ARG for s in causal_calls(L, r, **bad)), bad
    r = ctypes.byref(scan())
    for bad in (dict(u=None), dict(A=None), dict(Bm=None), dict(y=None), dict(u=OK + 2), dict(A=OK + 2), dict(Bm=OK + 1), dict(z=OK + 2),
                dict(D=OK + 1), dict(y=OK + 2), dict(state=OK + 2), dict(saved=OK + 8), dict(lengths=OK + 2)):
        assert all(s == B.GCONV_ERR_INVALID_ARG for s in scan_calls(L, r, **bad)), bad
    # a gradient of the gate without a gate, and the reverse; nothing saved
    tail = (OK, None, OK, BIG, None)
    assert L.gconv_scan_bwd(r, 0, OK, OK, OK, OK, OK, None, None, None, None, OK, OK, None, OK, OK, OK, OK, OK, None, OK, *tail) == \
        B.GCONV_ERR_INVALID_ARG
    assert L.gconv_scan_bwd(r, 0, OK, OK, OK, OK, OK, None, OK, None, None, OK, OK, None, OK, OK, OK, OK, OK, None, None, *tail) == \
        B.GCONV_ERR_INVALID_ARG
    assert L.gconv_scan_bwd(r, 0, OK, OK, OK, OK, OK, None, None, None, None, None, OK, None, OK, OK, OK, OK, OK, None, None, *tail) == \
        B.GCONV_ERR_INVALID_ARG


def test_workspaces(L):
    r = ctypes.byref(causal())
    need = L.gconv_causal_workspace_size(r, 0)
    assert 0 < need < 1 << 24
    for ws, n in ((None, BIG), (OK, need - 1), (OK + 4, BIG)):
        assert L.gconv_causal_bwd(r, 0, OK, OK, None, None, None, OK, None, OK, OK, None, None, ws, n, None) == B.GCONV_ERR_WORKSPACE
    r = ctypes.byref(scan())
    need = L.gconv_scan_workspace_size(r, 0, 1)
    assert need > 0
    for ws, n in ((None, BIG), (OK, need - 1), (OK + 4, BIG)):
        assert L.gconv_scan_bwd(r, 0, OK, OK, OK, OK, OK, None, None, None, None, OK, OK, None, OK, OK, OK, OK, OK, None, None, None, None,
                                ws, n, None) == B.GCONV_ERR_WORKSPACE


def test_saved_sizes(L):
    for n, c, l, s in ((2, 8, 30, 16), (1, 3, 65, 5), (3, 7, 64, 256)):
        for dt, es in ((0, 4), (1, 2)):
            marks = (n * -(-l // 64) * s * c * 4 + 15) // 16 * 16
            assert gc.gconv_scan_saved_size((n, c, l), s, dt) == marks
            assert gc.gconv_scan_saved_size((n, c, 1, l), s, dt, gated=True) == marks + n * c * l * es


def test_empty_batch(L):
    r = ctypes.byref(causal(N=0))
    assert L.gconv_causal_workspace_size(r, 0) == 0
    assert L.gconv_causal_fwd(r, 0, None, None, None, None, None, None, None, None) == B.GCONV_OK
    r = ctypes.byref(scan(N=0))
    assert L.gconv_scan_saved_size(r, 0, 1) == 0 and L.gconv_scan_workspace_size(r, 1, 1) == 0
    assert L.gconv_scan_fwd(r, 1, *[None] * 14, 0, None) == B.GCONV_OK


def test_binding_refusals():
    x, w = torch.zeros(2, 8, 30), torch.zeros(8, 4)
    with pytest.raises(ValueError):
        gc.gconv_causal_fwd(x, w, None, x)                         # no CUDA tensors
    with pytest.raises(TypeError):
        gc.gconv_causal_fwd(x.half(), w, None, x)
    with pytest.raises(ValueError):
        gc.gconv_causal_fwd(x, torch.zeros(7, 4), None, x)
    with pytest.raises(ValueError):
        gc.gconv_causal_fwd(torch.zeros(8), w, None, x)
    A, Bm = torch.zeros(8, 16), torch.zeros(2, 16, 30)
    with pytest.raises(ValueError):
        gc.gconv_scan_fwd(x, x, A, Bm, Bm, x)
    with pytest.raises(ValueError):
        gc.gconv_scan_fwd(x, x, A, torch.zeros(2, 15, 30), Bm, x)
    with pytest.raises(B.GconvError):
        gc.gconv_scan_saved_size((2, 8, 30), 300, 0)


@pytest.mark.parametrize("n", [0, 2])
def test_shapes_of_B(L, n):
    def look(shape, x=(n, 8, 5, 6), states=16, groups=2):
        return B._scan_record(torch.Size(x), torch.Size(shape), states, groups, 1, (0,) * 12, 0, 0)
    for shape in ((n, 32, 30), (n, 32, 5, 6), (n, 2, 16, 30), (n, 2, 16, 5, 6)):
        assert look(shape)[0].states == 16
    assert look((n, 32), (n, 8))[0].L == 1 and look((n, 2, 16), (n, 8))[0].L == 1
    # as many elements, but not a channel's positions one behind the other
    for shape in ((n, 30, 32), (n, 16, 2, 30), (n, 30, 2, 16), (n, 32, 29), (n, 32), (n, 960), (32, n, 30), (n,)):
        with pytest.raises(ValueError):
            look(shape)
