"""Forms of the paged calls that the other tests' sizes do not reach: many KV heads, every group size with
masses at both head sizes, long appends and gathers of every type and head size."""
import numpy as np
import pytest
import torch

import attention_scored_kv_gb300 as kvs
from oracle import paged as ref
from tests.test_gpu_paged import DT, check_mass, check_out, f64, filled, i32, make, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 7, 8, 9, 16, 17, 31, 32, 33])
def test_groups_with_masses(group, d):
    kv = [700, 0, 129, 1]
    cache, orc, table, q = filled(kv, [1] * 4, 2 * group, 2, d, kvs.BF16, seed=group)
    want = orc.attend(f64(q), table, kv)
    mass = torch.full(table.shape, -3.0, device="cuda")
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), block_mass=mass)
    check_out(out, want, d, kvs.BF16, True)
    check_mass(mass, want, np.arange(table.shape[1])[None] >= -(-np.asarray(kv)[:, None] // 16), d)
    assert cache.get_status() == 0


@pytest.mark.parametrize("hq,hkv,d,new", [(64, 64, 64, 1), (512, 512, 64, 1), (1024, 1024, 64, 3), (192, 96, 128, 2), (96, 96, 128, 40)])
def test_many_kv_heads(hq, hkv, d, new):
    kv = [150, 40]
    cache, orc, table, q = filled(kv, [new, new], hq, hkv, d, kvs.BF16, seed=hkv)
    start = [0, new, 2 * new]
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=new)
    check_out(out, orc.attend(f64(q), table, kv, start), d, kvs.BF16, True)
    assert cache.get_status() == 0


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
def test_long_appends_and_gathers(d, dt):
    """Sixteen rows to a warp; rows read in order, from the middle of pages, backwards and at random."""
    g, rng = torch.Generator().manual_seed(d), np.random.default_rng(d)
    lens = [7, 3001, 1990, 16]
    blocks = [-(-n // 16) for n in lens]
    pages = sum(blocks)
    cache, orc = make(hq=1, hkv=1, d=d, pages=pages, dt=dt), ref.Pages(pages, 1, d)
    perm, at, slots = rng.permutation(pages), 0, []
    for n, b in zip(lens, blocks):
        p = np.arange(n)
        slots.append(perm[at:at + b][p // 16] * 16 + p % 16)
        at += b
    first, rest = [s[:n // 3] for s, n in zip(slots, lens)], [s[n // 3:] for s, n in zip(slots, lens)]
    for part in (first, rest):                             # the second call joins pages that the first one began
        s = np.concatenate(part + [np.full(5, -1)] + ([np.full(4200, -1)] if len(np.concatenate(part)) < 4097 else []))
        k, v = rand(g, (len(s), 1, d), dt, 2.0), rand(g, (len(s), 1, d), dt, 0.5)
        cache.append(0, k.cuda(), v.cuda(), i32(s))
        orc.append(f64(k), f64(v), s)
    every = np.concatenate(slots)
    for want in (every, every[5:], every[::-1].copy(), rng.permutation(every), np.concatenate([every[3000:], [-1] * 20, every[:3000]])):
        assert len(want) * 2 > 8192
        for x, y in zip(cache.gather(0, i32(want)), orc.gather(want)):
            assert x.dtype == DT[dt] and np.array_equal(f64(x), y)
    assert cache.get_status() == 0
