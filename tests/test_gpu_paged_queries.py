"""Queries in which one element is far larger than the others, which alone decide the weights
(K is 0 where the large one is, as for a channel that only some heads use).

The kernels split a bf16 query into two 8-bit floats, exact for elements down to 2^-13 of the
largest: the tolerance is the usual one of test_gpu_paged_weights.py, without a term for it.
Below that an element may be off by 2^-21 of the largest; a logit is then off by
2^-21 max|q| sum_d |k_d| / sqrt(D), which that test adds to delta.
"""
import numpy as np
import pytest
import torch

import attention_scored_kv_gb300 as kvs
from tests.test_gpu_paged import f64, i32, stored
from tests.test_gpu_paged_weights import exact

pytestmark = pytest.mark.gpu

FORMS = [(8, 1), (8, 2), (16, 1), (8, 4), (64, 1), (8, 40), (32, 9)]


def attend(ctx, q, k, v, hq, d, rows):
    cache, orc, table = stored([ctx], k, v, d, hq, 1, 7)
    out = cache.attend(0, q.cuda(), i32(table), i32([ctx]), q_start=i32([0, rows]), max_q_len=rows)
    assert cache.get_status() == 0
    slots = table[0, np.arange(ctx) // 16] * 16 + np.arange(ctx) % 16
    return out, exact(orc, table, ctx, q), orc.gather(slots)[0][:, 0]


def check(out, want, few, more=0.0):
    o, spread, floor, reach, _ = want
    d = o.shape[2]
    delta = (d + 8) * 2.0 ** -23 * reach + 2.0 ** -21 * (1 + reach) + more
    tol = 2.0 ** -8 * np.abs(o) + ((2.0 ** -11 if few else 2.0 ** -8) + 2.0 ** -19 + 4 * delta[:, :, None]) * spread
    tol += (2.0 ** -38 if few else 0.0) * floor
    err = np.abs(f64(out) - o)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("hq,rows", FORMS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("large", [2048.0, -4096.0])
def test_small_elements_are_exact(large, d, hq, rows):
    ctx, g = 900, torch.Generator().manual_seed(d + hq + rows)
    q = torch.full((rows, hq, d), 1 + 2.0 ** -7)           # its last bit is what a short second piece would drop
    q[..., 0] = large
    k = 3 * (2 * torch.rand((ctx, 1, 1), generator=g) - 1) + 0.3 * torch.randn((ctx, 1, d), generator=g)
    k[..., 0] = 0
    v = torch.randn((ctx, 1, d), generator=g)
    out, want, _ = attend(ctx, q.bfloat16(), k.bfloat16(), v.bfloat16(), hq, d, rows)
    check(out, want, hq * rows <= 16)


@pytest.mark.parametrize("hq,rows", FORMS)
@pytest.mark.parametrize("large", [2.0 ** 14, 2.0 ** 17])
def test_smaller_ones_are_close(large, hq, rows):
    ctx, d, g = 900, 128, torch.Generator().manual_seed(hq + rows)
    q = torch.randn((rows, hq, d), generator=g)
    q[..., 5] = large
    k, v = (torch.randn((ctx, 1, d), generator=g) for _ in range(2))
    k[..., 5] = 0
    out, want, kd = attend(ctx, q.bfloat16(), k.bfloat16(), v.bfloat16(), hq, d, rows)
    check(out, want, hq * rows <= 16, more=2.0 ** -21 * large * np.abs(kd).sum(1).max() / d ** 0.5)
