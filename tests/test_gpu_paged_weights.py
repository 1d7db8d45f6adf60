"""The paged attends on rows whose output is made of small weights: one token takes nearly
all of the weight and has the value 0 in a page of ordinary ones, as a head's attention sink
does, so that what is left is the sum of very many weights of 2^-10 to 2^-40 of it.

Tolerance per output element, all from the exact weights a_j in 64 bits, with A = sum_j a_j
|v_j|, u = eps/2 of the output type and delta as in test_gpu_paged.py (a logit's error):

  |o - o*| <= u |o*| + (r + 2^-19 + 4 delta) A + 2^-38 T

  r: what a probability is rounded to before its product with V: 2^-11 in the single-token
  kernel (three pieces of 3 significant bits), 2^-8 in the prompt kernel (bf16, and as much
  in the sum that it is divided by), 2^-23 on the CUDA cores.
  2^-19: the float32 sums of the products, each addition off by 2^-23 of the magnitudes at
  most, 128 tokens of a tile and the pieces' and tiles' sums together less than 16 of them at
  a time in the tensor core.
  T, single-token kernel only: a probability has those bits down to the smallest step of the
  last piece, which is 2^-38 of the tile's heaviest a_j * (V scale): T = sum over tiles of
  max_j(a_j * V scale) sum_j |V code|.
"""
import functools
import math

import numpy as np
import pytest
import torch

import attention_scored_kv_gb300 as kvs
from tests.test_gpu_paged import DT, f64, i32, stored

pytestmark = pytest.mark.gpu


def sink_case(ctx, weight, sigma, hq, d, rows, seed):
    """K, V [ctx, 1, d] and queries [rows, hq, d]: token 3 is the sink of every row."""
    g = torch.Generator().manual_seed(seed)
    sign = torch.sign(torch.randn((1, 1, d), generator=g))
    q = (sign + 0.05 * torch.randn((rows, hq, d), generator=g)).to(torch.bfloat16)
    k = sigma * torch.randn((ctx, 1, d), generator=g)
    logit = math.log(ctx) + sigma * sigma / 2 + math.log(weight / (1 - weight))
    k[3] = logit / math.sqrt(d) * sign[0]
    v = 1 + 0.5 * torch.randn((ctx, 1, d), generator=g)
    v[3] = 0
    return k.to(torch.bfloat16), v.to(torch.bfloat16), q


def exact(orc, table, kv, q, window=0):
    """out, A, T, delta's reach of the rows of one request of one KV head, and the blocks' masses of its last row."""
    slots = table[0, np.arange(kv) // 16] * 16 + np.arange(kv) % 16
    k, v = (x[:, 0] for x in orc.gather(slots))
    vs = orc.scales[1][table[0], 0].repeat(16)[:kv]
    rows, hq, d = q.shape
    out, spread, floor = np.zeros((rows, hq, d)), np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    reach, mass = np.zeros((rows, hq)), np.zeros(-(-kv // 16))
    for i in range(rows):
        hi = kv - rows + i + 1
        lo = max(hi - window, 0) if window else 0
        first = (max(kv - rows + 1 - window, 0) if window else 0) // 16 * 16     # where the request's tiles start
        s = f64(q[i]) @ k[lo:hi].T / math.sqrt(d)
        reach[i] = (np.abs(f64(q[i])) @ np.abs(k[lo:hi]).T).max(-1) / math.sqrt(d)
        a = np.exp(s - s.max(-1, keepdims=True))
        a /= a.sum(-1, keepdims=True)
        out[i], spread[i] = a @ v[lo:hi], a @ np.abs(v[lo:hi])
        cuts = np.unique(np.concatenate([[0], (np.arange(first, hi, 128) - lo).clip(0)]))
        cuts = cuts[cuts < hi - lo]
        top = np.maximum.reduceat(a * vs[lo:hi], cuts, axis=1)
        floor[i] = top @ np.add.reduceat(np.abs(v[lo:hi]) / vs[lo:hi, None], cuts, axis=0)
        blocks = np.zeros((hq, len(mass)))
        np.add.at(blocks.T, np.arange(lo, hi) // 16, a.T)
        mass = blocks.max(0)
    return out, spread, floor, reach, mass


def check(out, want, d, dt, r, smallest):
    o, spread, floor, reach, _ = want
    delta = (d + 8) * 2.0 ** -23 * reach + 2.0 ** -21 * (1 + reach)
    tol = torch.finfo(DT[dt]).eps / 2 * np.abs(o) + (r + 2.0 ** -19 + 4 * delta[:, :, None]) * spread + smallest * floor
    err = np.abs(f64(out) - o)
    assert (err <= tol).all(), ((err / tol).max(), (err / np.abs(o)).max())


@functools.lru_cache(maxsize=1)
def sink_oracle(ctx, weight, sigma, d):
    k, v, q = sink_case(ctx, weight, sigma, 64, d, 40, seed=d)
    _, orc, table = stored([ctx], k, v, d, 64, 1, 7)
    return k, v, q, orc, table


SINKS = [(100, 0.99, 1.0), (128, 0.9999, 1.0), (1000, 0.9999, 1.0), (5000, 0.999, 2.0), (32768, 0.99, 1.0),
         (32768, 0.999, 1.0), (131072, 0.99, 0.5), (131072, 0.9999, 0.5), (131072, 0.99, 2.0)]


# a group of 8 with one and two rows, of 16, and of 64 (the prompt kernel); few rows and prompt rows
@pytest.mark.parametrize("hq,rows", [(8, 1), (8, 2), (16, 1), (8, 4), (64, 1), (8, 40)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctx,weight,sigma", SINKS)
def test_sinks_without_value(ctx, weight, sigma, d, hq, rows):
    if rows == 40 and ctx > 5000:
        rows = 20
    k, v, q, orc, table = sink_oracle(ctx, weight, sigma, d)
    q = q[:rows, :hq].contiguous()
    cache = kvs.PagedCache(kvs.paged_config_init(num_layers=1, num_q_heads=hq, num_kv_heads=1, head_dim=d,
                                                 num_pages=orc.num_pages))
    cache.append(0, k.cuda(), v.cuda(), i32(table[0, np.arange(ctx) // 16] * 16 + np.arange(ctx) % 16))
    want = exact(orc, table, ctx, q)
    out = cache.attend(0, q.cuda(), i32(table), i32([ctx]), q_start=i32([0, rows]), max_q_len=rows)
    if hq * rows <= 16:
        check(out, want, d, kvs.BF16, 2.0 ** -11, 2.0 ** -38)
    else:
        check(out, want, d, kvs.BF16, 2.0 ** -8, 0.0)
    assert cache.get_status() == 0


@pytest.mark.parametrize("hq", [8, 16, 32])
@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("ctx,weight,sigma", [(600, 0.9999, 1.0), (32768, 0.999, 1.0)])
def test_sinks_with_masses(ctx, weight, sigma, window, hq):
    d = 128
    k, v, q = sink_case(ctx, weight, sigma, hq, d, 1, seed=hq)
    if window:                                   # the sink within the window
        k[[3, ctx - 300]], v[[3, ctx - 300]] = k[[ctx - 300, 3]], v[[ctx - 300, 3]]
    cache, orc, table = stored([ctx], k, v, d, hq, 1, 7)
    want = exact(orc, table, ctx, q, window)
    mass = torch.full(table.shape, -3.0, device="cuda")
    out = cache.attend(0, q.cuda(), i32(table), i32([ctx]), window=window, block_mass=mass)
    check(out, want, d, kvs.BF16, 2.0 ** -11, 2.0 ** -38)
    reach = want[3].max()
    delta = (d + 8) * 2.0 ** -23 * reach + 2.0 ** -21 * (1 + reach)
    first = max(ctx - window, 0) // 16 if window else 0
    assert (f64(mass)[0, :first] == -3.0).all()
    assert (np.abs(f64(mass)[0, first:] - want[4][first:]) <= 8 * delta * want[4][first:] + 1e-30).all()
    assert cache.get_status() == 0


@pytest.mark.parametrize("rows", [1, 3])
def test_sinks_in_float32(rows):
    ctx, d, hq = 3000, 128, 8
    k, v, q = sink_case(ctx, 0.9999, 1.0, hq, d, rows, seed=rows)
    cache, orc, table = stored([ctx], k, v, d, hq, 1, 7)
    wide = kvs.PagedCache(kvs.paged_config_init(num_layers=1, num_q_heads=hq, num_kv_heads=1, head_dim=d,
                                                num_pages=cache.cfg.num_pages, in_dtype=kvs.F32))
    slots = i32(table[0, np.arange(ctx) // 16] * 16 + np.arange(ctx) % 16)
    wide.append(0, k.float().cuda(), v.float().cuda(), slots)
    out = wide.attend(0, q.float().cuda(), i32(table), i32([ctx]), q_start=i32([0, rows]), max_q_len=rows)
    check(out, exact(orc, table, ctx, q), d, kvs.F32, 2.0 ** -23, 0.0)


@pytest.mark.parametrize("hq,kernel", [(8, kvs.KERNEL_AUTO), (32, kvs.KERNEL_AUTO), (8, kvs.KERNEL_GENERAL)])
def test_masses_leave_out_heads_that_are_not_finite(hq, kernel):
    """The others' masses are as before; where no head is finite they are 0."""
    ctx, d = 900, 128
    g = torch.Generator().manual_seed(hq)
    k, v = (torch.randn((2 * ctx, 1, d), generator=g).bfloat16() for _ in range(2))
    q = torch.randn((2, hq, d), generator=g).bfloat16()
    cache, orc, table = stored([ctx, ctx], k, v, d, hq, 1, 7)
    if kernel == kvs.KERNEL_GENERAL:
        cache = kvs.PagedCache(kvs.paged_config_init(num_layers=1, num_q_heads=hq, num_kv_heads=1, head_dim=d,
                                                     num_pages=cache.cfg.num_pages, kernel=kernel))
        slots = np.concatenate([table[r, np.arange(ctx) // 16] * 16 + np.arange(ctx) % 16 for r in range(2)])
        cache.append(0, k.cuda(), v.cuda(), i32(slots))
    bad = q.clone()
    bad[0, 1, 5], bad[0, 4, 100] = float("nan"), float("-inf")
    bad[1, :, 0] = float("inf")
    mass = torch.full(table.shape, -3.0, device="cuda")
    out = cache.attend(0, bad.cuda(), i32(table), i32([ctx, ctx]), block_mass=mass)
    keep = [h for h in range(hq) if h not in (1, 4)]
    want = orc.attend(f64(q[:1, keep]), table[:1], [ctx])
    reach = want["reach"].max()
    delta = (d + 8) * 2.0 ** -23 * reach + 2.0 ** -21 * (1 + reach)
    assert (np.abs(f64(mass)[0] - want["mass"][0]) <= 8 * delta * want["mass"][0] + 1e-30).all()
    assert (mass[1] == 0).all() and out[1].isnan().all() and out[0, 1].isnan().all()
    assert out[0, keep].isfinite().all() and cache.get_status() == 0
