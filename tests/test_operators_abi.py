"""Block and orthogonalisation entry points without a GPU: sizes and refusals, none of which
reaches a launch."""
import ctypes

import pytest

from bwd_gconv_fwd_gb300 import binding as B

BAD = ctypes.c_size_t(-1).value
OK = 1 << 20      # an aligned address that is never touched
ODD = OK + 2


@pytest.fixture(scope="module")
def L():
    from bwd_gconv_fwd_gb300 import build
    build.build()
    return B.lib()


def block(N=2, C=8, H=3, W=3, groups=1, eps=1e-6, gate=0, act=0):
    return B.Block(N, C, H, W, groups, eps, gate, act)


WRONG = [block(N=-1), block(C=0), block(H=0), block(W=0), block(groups=0), block(groups=3), block(eps=-1.0),
         block(eps=float("nan")), block(eps=float("inf")), block(gate=3), block(gate=-1), block(act=3),
         block(N=70000, C=4096, H=100, W=100)]


@pytest.mark.parametrize("b", WRONG)
def test_invalid_block_records(L, b):
    r = ctypes.byref(b)
    assert L.gconv_block_workspace_size(r, B.GCONV_F32) == BAD
    assert L.gconv_norm_fwd(r, 0, OK, None, OK, None) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_norm_bwd(r, 0, OK, None, OK, None, OK, None, OK, 1 << 30, None) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_join_fwd(r, 0, OK, OK, None, None, None, None, OK, None, None) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_join_bwd(r, 0, None, OK, None, None, None, None, OK, None, None, OK, None, None, None, None, OK, 1 << 30,
                            None) == B.GCONV_ERR_INVALID_ARG


def test_null_record_and_dtype(L):
    assert L.gconv_block_workspace_size(None, 0) == BAD
    assert L.gconv_block_workspace_size(ctypes.byref(block()), 2) == BAD
    assert L.gconv_norm_fwd(None, 0, OK, None, OK, None) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_orthogonalize_workspace_size(None) == BAD


def test_block_pointers(L):
    r = ctypes.byref(block())
    big = 1 << 30
    for x, y in ((None, OK), (OK, None), (ODD, OK), (OK, ODD)):
        assert L.gconv_norm_fwd(r, 0, x, None, y, None) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_norm_fwd(r, 0, OK, ODD, OK, None) == B.GCONV_ERR_INVALID_ARG
    need = L.gconv_block_workspace_size(r, 0)
    assert 0 < need < 1 << 20
    assert L.gconv_norm_bwd(r, 0, OK, None, OK, None, OK, None, OK, need - 1, None) == B.GCONV_ERR_WORKSPACE
    assert L.gconv_norm_bwd(r, 0, OK, None, OK, None, OK, None, None, big, None) == B.GCONV_ERR_WORKSPACE
    assert L.gconv_norm_bwd(r, 0, OK, None, None, None, OK, None, OK, big, None) == B.GCONV_ERR_INVALID_ARG
    # a gate that the record does not announce, and the reverse; next_weight without next
    assert L.gconv_join_fwd(r, 0, OK, OK, OK, None, None, None, OK, None, None) == B.GCONV_ERR_INVALID_ARG
    gated = ctypes.byref(block(gate=1))
    assert L.gconv_join_fwd(gated, 0, OK, OK, None, None, None, None, OK, None, None) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_join_fwd(r, 0, OK, OK, None, None, None, OK, OK, None, None) == B.GCONV_ERR_INVALID_ARG
    # backward: neither gradient; a next without out or dres; dres without a next; dgate without a gate
    tail = (OK, None, None, None, None, OK, big, None)
    assert L.gconv_join_bwd(r, 0, OK, OK, None, None, None, None, None, None, None, *tail) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_join_bwd(r, 0, None, OK, None, None, None, None, OK, OK, OK, *tail) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_join_bwd(r, 0, OK, OK, None, None, None, None, OK, OK, None, *tail) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_join_bwd(r, 0, OK, OK, None, None, None, None, OK, None, OK, *tail) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_join_bwd(r, 0, None, OK, None, None, None, None, OK, None, None, OK, OK, None, None, None, OK, big,
                            None) == B.GCONV_ERR_INVALID_ARG


def test_empty_batch(L):
    r = ctypes.byref(block(N=0))
    assert L.gconv_block_workspace_size(r, 0) == 0
    assert L.gconv_norm_fwd(r, 0, None, None, None, None) == B.GCONV_OK
    assert L.gconv_norm_bwd(r, 0, None, None, None, None, None, None, None, 0, None) == B.GCONV_OK
    assert L.gconv_join_fwd(r, 1, None, None, None, None, None, None, None, None, None) == B.GCONV_OK


@pytest.mark.parametrize("count,rows,cols", [(-1, 4, 4), (1, 0, 4), (1, 4, 0), (1, 1 << 16, 1 << 16), (3, 1 << 15, 1 << 15)])
def test_invalid_matrices(L, count, rows, cols):
    m = ctypes.byref(B.Matrices(count, rows, cols))
    assert L.gconv_orthogonalize_workspace_size(m) == BAD
    assert L.gconv_orthogonalize(m, 0, 0, OK, OK, 5, None, 0.0, OK, 1 << 40, None) == B.GCONV_ERR_INVALID_ARG


def test_orthogonalize_arguments(L):
    m = ctypes.byref(B.Matrices(1, 300, 400))
    need = L.gconv_orthogonalize_workspace_size(m)
    assert need > 300 * 400 * 2 * 2
    nan = (ctypes.c_float * 3)(1.0, float("nan"), 0.0)
    call = lambda g=OK, out=OK, steps=5, c=None, eps=1e-7, ws=OK, n=need, dt=0, odt=0: \
        L.gconv_orthogonalize(m, dt, odt, g, out, steps, c, eps, ws, n, None)  # noqa: E731
    for bad in (dict(steps=0), dict(steps=65), dict(c=nan, steps=1), dict(eps=-1.0), dict(eps=float("nan")), dict(g=None),
                dict(out=None), dict(g=ODD), dict(out=ODD), dict(ws=ODD), dict(dt=2), dict(odt=-1)):
        assert call(**bad) in (B.GCONV_ERR_INVALID_ARG, B.GCONV_ERR_WORKSPACE), bad
    empty = ctypes.byref(B.Matrices(0, 300, 400))
    assert L.gconv_orthogonalize_workspace_size(empty) == 0
    assert L.gconv_orthogonalize(empty, 0, 0, None, None, 5, None, 0.0, None, 0, None) == B.GCONV_OK


def test_muon_arguments(L):
    m = ctypes.byref(B.Matrices(2, 8, 18))
    for kw in (dict(lr=float("nan")), dict(beta=float("inf")), dict(weight_decay=float("nan")), dict(steps=0)):
        v = dict(lr=0.1, beta=0.9, weight_decay=0.0, scale=0.0, eps=1e-7, nesterov=1, steps=5) | kw
        opt = ctypes.byref(B.Muon(*v.values(), None))
        assert L.gconv_muon_step(m, opt, OK, OK, OK, OK, OK, None, OK, 1 << 30, None) == B.GCONV_ERR_INVALID_ARG
    opt = ctypes.byref(B.Muon(0.1, 0.9, 0.0, 0.0, 1e-7, 1, 5, None))
    for k in range(5):
        p = [OK] * 5
        for wrong in (None, ODD):
            p[k] = wrong
            assert L.gconv_muon_step(m, opt, *p, None, OK, 1 << 30, None) == B.GCONV_ERR_INVALID_ARG
    assert L.gconv_muon_step(m, None, OK, OK, OK, OK, OK, None, OK, 1 << 30, None) == B.GCONV_ERR_INVALID_ARG


def test_sizes_are_kept_by_device(monkeypatch):
    """Workspace sizes depend on the device's number of SMs: what was asked on one is not taken for another."""
    torch = pytest.importorskip("torch")
    now = [0]

    class Fake:
        def gconv_block_workspace_size(self, block, dt):
            return 1000 + now[0]

        def gconv_orthogonalize_workspace_size(self, matrices):
            return 2000 + now[0]

    monkeypatch.setattr(B, "_lib", Fake())
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    for k in (B._block_record, B._matrices):
        k.cache_clear()
    try:
        for device in (0, 1, 0):
            now[0] = device
            assert B.gconv_block_workspace_size((2, 8, 3, 3), B.GCONV_F32) == 1000 + device
            assert B.gconv_orthogonalize_workspace_size((300, 400)) == 2000 + device
    finally:
        for k in (B._block_record, B._matrices):
            k.cache_clear()
