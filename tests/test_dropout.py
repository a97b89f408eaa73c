"""Dropout: the generator against its published vectors, the kernel against the definition, refusals."""
import numpy as np
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from bwd_gconv_fwd_gb300 import binding as B

M32 = np.uint64(0xFFFFFFFF)


def philox(counter, key):
    """Philox-4x32-10 of Salmon et al., 2011: counter four and key two 32-bit words, arrays of uint64."""
    c, k = [np.asarray(v, dtype=np.uint64) for v in counter], [np.uint64(v) for v in key]
    for _ in range(10):
        p, q = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(q >> np.uint64(32)) ^ c[1] ^ k[0], q & M32, (p >> np.uint64(32)) ^ c[3] ^ k[1], p & M32]
        k = [(k[0] + np.uint64(0x9E3779B9)) & M32, (k[1] + np.uint64(0xBB67AE85)) & M32]
    return c


def keep(count, seed, step, p):
    seed, step = seed % 2 ** 64, step % 2 ** 64
    i = np.arange((count + 3) // 4, dtype=np.uint64)
    full = lambda v: np.full_like(i, v)  # noqa: E731
    w = philox([i & M32, i >> np.uint64(32), full(step & 0xFFFFFFFF), full(step >> 32)], [seed & 0xFFFFFFFF, seed >> 32])
    return np.stack(w, 1).reshape(-1)[:count] >= np.uint64(int(p * 2.0 ** 32))


def test_generator_vectors():
    """The generator's published answers at counters and keys of all zeros and all ones."""
    zero, ones = [np.zeros(1, np.uint64)] * 4, [np.full(1, 0xFFFFFFFF, np.uint64)] * 4
    assert [int(v[0]) for v in philox(zero, [0, 0])] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert [int(v[0]) for v in philox(ones, [0xFFFFFFFF] * 2)] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_refusals():
    from bwd_gconv_fwd_gb300 import build
    build.build()
    L, ok = B.lib(), 1 << 20
    for p in (-0.1, 1.5, float("nan"), float("inf")):
        assert L.gconv_dropout_fwd(8, 0, ok, None, ok, p, ok, None) == B.GCONV_ERR_INVALID_ARG
        assert L.gconv_dropout_bwd(8, 0, ok, ok, p, ok, None) == B.GCONV_ERR_INVALID_ARG
    for args in ((-1, 0, ok, None, ok, 0.1, ok), (1 << 41, 0, ok, None, ok, 0.1, ok), (8, 2, ok, None, ok, 0.1, ok),
                 (8, 0, None, None, ok, 0.1, ok), (8, 0, ok, None, None, 0.1, ok), (8, 0, ok, None, ok, 0.1, None),
                 (8, 0, ok + 2, None, ok, 0.1, ok), (8, 1, ok + 1, None, ok, 0.1, ok), (8, 0, ok, ok + 1, ok, 0.1, ok),
                 (8, 0, ok, None, ok + 4, 0.1, ok), (8, 0, ok, None, ok, 0.1, ok + 3)):
        assert L.gconv_dropout_fwd(*args, None) == B.GCONV_ERR_INVALID_ARG, args
    assert L.gconv_dropout_fwd(0, 0, None, None, None, 0.1, None, None) == B.GCONV_OK
    x = torch.zeros(4)
    with pytest.raises(ValueError):
        gc.gconv_dropout_fwd(x, x, torch.zeros(2, dtype=torch.int64), 0.1)
    with pytest.raises(TypeError):
        gc.gconv_dropout_fwd(x.half(), x.half(), torch.zeros(2, dtype=torch.int64), 0.1)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_gconv_fwd_gb300 import build
    build.build()
    return torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("count,offset", [(1, 0), (3, 0), (4, 1), (7, 0), (8, 0), (9, 3), (1000, 0), (2048, 2), (2049, 0), (100003, 0), (65536, 1)])
def test_dropout(dev, count, offset, dtype):
    gen = torch.Generator().manual_seed(count)
    for p, seed, step in ((0.1, 5, 7), (0.5, -3, 2 ** 40 + 1), (0.0, 1, 1), (1.0, 1, 1), (0.9, 2 ** 62, -1)):
        big = torch.randn((3, count + offset), generator=gen).to(dtype).to(dev)
        x, res = (big[i].clone()[offset:] for i in range(2))
        if count > 20:
            x[::7] = float("nan")
            x[3::7] = float("inf")
        rng = torch.tensor([seed, step], dtype=torch.int64, device=dev)
        guard = torch.full((count + offset + 64,), 7.5, dtype=dtype, device=dev)
        y = guard[offset:offset + count]
        gc.gconv_dropout_fwd(x, y, rng, p, res=res)
        mask = torch.from_numpy(keep(count, seed, step, p) if p < 1 else np.zeros(count, bool)).to(dev)
        scale = 0.0 if p == 1 else 2.0 ** 32 / (2.0 ** 32 - int(p * 2.0 ** 32))
        ref = torch.where(mask, x.double() * scale, 0.0)

        def same(got, want):
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            fine = torch.isfinite(want)
            assert torch.equal(got.double()[torch.isinf(want)], want[torch.isinf(want)])
            g, w = got.double()[fine], want[fine]
            # the scale is rounded to fp32, the product and the sum once each (x scale is at most w + res), then dtype
            size = w.abs() + (res.double()[fine].abs() * 2 if want is not ref else 0)
            assert bool(((g - w).abs() <= 2.0 ** -22 * size + (2.0 ** -8 * w.abs() if dtype == torch.bfloat16 else 0)).all())

        same(y, ref + res.double())
        assert bool((guard[:offset] == 7.5).all()) and bool((guard[offset + count:] == 7.5).all())
        dx = torch.empty_like(x)
        gc.gconv_dropout_bwd(x, dx, rng, p)
        same(dx, ref)
        gc.gconv_dropout_fwd(x, x, rng, p)          # in place
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(dx))


@pytest.mark.gpu
def test_replays_draw_new_masks(dev):
    x, y = torch.ones(5000, device=dev), torch.empty(5000, device=dev)
    rng = torch.tensor([9, 0], device=dev)
    gc.gconv_dropout_fwd(x, y, rng, 0.3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gc.gconv_dropout_fwd(x, y, rng, 0.3)
        rng[1] += 1
    for step in range(3):
        graph.replay()
        assert torch.equal(y != 0, torch.from_numpy(keep(5000, 9, step, 0.3)).to(dev))


@pytest.mark.gpu
def test_beyond_32_bits(dev):
    """More than 2^32 elements: counters and addresses of the last ones."""
    count = 2 ** 32 + 12345
    if torch.cuda.get_device_properties(dev).total_memory < 6 * count:
        pytest.skip("needs 26 GB")
    x = torch.ones(count, dtype=torch.bfloat16, device=dev)
    rng = torch.tensor([1, 2], device=dev)
    gc.gconv_dropout_fwd(x, x, rng, 0.5)
    tail = 20001
    i = np.arange((count - tail) // 4, (count + 3) // 4, dtype=np.uint64)
    w = np.stack(philox([i & M32, i >> np.uint64(32), np.full_like(i, 2), np.full_like(i, 0)], [1, 0]), 1).reshape(-1)
    w = w[(count - tail) % 4:][:tail]
    assert torch.equal(x[count - tail:] != 0, torch.from_numpy(w >= np.uint64(2 ** 31)).to(dev))
