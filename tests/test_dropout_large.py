"""Dropout at the sizes of its main kernel: at least a tile of 512 16-byte pieces for every multiprocessor."""
import numpy as np
import pytest
import torch

import bwd_gconv_fwd_gb300 as gc
from test_dropout import dev, keep  # noqa: F401

pytestmark = pytest.mark.gpu


def same(got, want, size, dtype):
    """NaN and infinities as they are; the scale, the product and the sum are rounded to fp32 once each, then dtype."""
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    inf, fine = torch.isinf(want), torch.isfinite(want)
    assert torch.equal(got.double()[inf], want[inf])
    g, w = got.double()[fine], want[fine]
    assert bool(((g - w).abs() <= 2.0 ** -22 * size[fine] + (2.0 ** -8 * w.abs() if dtype == torch.bfloat16 else 0)).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])             # on 16 bytes, and off them: the kernel of small sizes at the same ones
# whole tiles, and elements behind the last of them: one round of the first blocks, and five rounds and a few tiles more
@pytest.mark.parametrize("rounds,tiles,rest", [(1, 0, 0), (1, 0, 3), (1, 1, 1027), (5, 7, 2046), (9, 3, 1)])
def test_large(dev, rounds, tiles, rest, offset, dtype):  # noqa: F811
    tile = 512 * 16 // (2 if dtype == torch.bfloat16 else 4)
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    count = (rounds * sms + tiles) * tile + rest
    gen = torch.Generator(device=dev).manual_seed(count)
    x0, res0 = (torch.empty(count, device=dev).normal_(generator=gen).to(dtype) for _ in range(2))
    x0[::7], x0[3::7] = float("nan"), float("inf")

    def placed(t):
        """The same values at the offset, between guard words."""
        buf = torch.full((count + offset + 64,), 7.5, dtype=dtype, device=dev)
        buf[offset:offset + count] = t
        return buf, buf[offset:offset + count]

    for p, seed, step in ((0.1, 5, 7), (0.3, -3, 2 ** 40 + 1), (0.0, 1, 1), (1.0, 1, 1), (0.9, 2 ** 62, -1)):
        rng = torch.tensor([seed, step], dtype=torch.int64, device=dev)
        mask = torch.from_numpy(keep(count, seed, step, p) if p < 1 else np.zeros(count, bool)).to(dev)
        scale = 0.0 if p == 1 else 2.0 ** 32 / (2.0 ** 32 - int(p * 2.0 ** 32))
        ref = torch.where(mask, x0.double() * scale, 0.0)
        both, size = ref + res0.double(), ref.abs() + 2 * res0.double().abs()
        (_, x), (_, res), (guard, y) = placed(x0), placed(res0), placed(torch.zeros_like(x0))
        gc.gconv_dropout_fwd(x, y, rng, p, res=res)
        same(y, both, size, dtype)
        gc.gconv_dropout_bwd(x, y, rng, p)
        same(y, ref, ref.abs(), dtype)
        plain = y.clone()
        gc.gconv_dropout_fwd(x, y, rng, p)
        assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(plain))
        assert bool((guard[:offset] == 7.5).all()) and bool((guard[offset + count:] == 7.5).all())
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(x0)) and torch.equal(res, res0)
        # in place: onto the residual, then onto x
        for i in (1, 0):
            (xg, x), (rg, res) = placed(x0), placed(res0)
            gc.gconv_dropout_fwd(x, res if i else x, rng, p, res=res)
            same(res if i else x, both, size, dtype)
            for g in (xg, rg):
                assert bool((g[:offset] == 7.5).all()) and bool((g[offset + count:] == 7.5).all())
        (xg, x) = placed(x0)
        gc.gconv_dropout_bwd(x, x, rng, p)
        assert torch.equal(torch.nan_to_num(x), torch.nan_to_num(plain))
        assert bool((xg[:offset] == 7.5).all()) and bool((xg[offset + count:] == 7.5).all())
