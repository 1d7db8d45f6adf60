"""The paged E4M3 cache on the GPU against its float64 oracle.

Tables, slots, codes and scales are exact (integers, or values rounded once by rules that
the oracle states), so they are compared for equality.  Attention tolerances, per output
element, with A = sum_j a_j |v_j| from the oracle and u = eps/2 of the output type
(half a step, relative):

  |o - o*| <= u |o*| + (r + 4 delta) A + 2^-23 F

  delta: a logit's error in nats.  Products of a query with a code are exact in float32; the
  D of them are summed in float32, each addition off by at most 2^-23 of the sum of the
  magnitudes so far (truncation at worst), then scaled: (D + 8) 2^-23 sum_d |q k| / sqrt(D),
  and exp2 and the subtraction of the maximum add 2^-21 (1 + |s|), |s| <= that sum.  A
  normalised probability is off by twice that relatively (itself and the sum), four times
  with the statistics' own rounding.
  r: what a probability is rounded to before its product with V: 2^-9 where it is kept in
  two 8-bit pieces of 4 significant bits each, 2^-9 in bf16 and as much in the sum that it is
  divided by, covered by 2^-8 for both; the float32 path keeps 2^-23 (D of its roundings are
  in delta's term).
  F: rounding is relative only down to the smallest step.  The tensor-core decode keeps x =
  a_j * (V scale), relative to its largest, as 2^8 at most; E4M3's smallest step is 2^-9 and
  the second piece carries a factor of 32, so x is off by up to 2^-15, 2^-23 of the largest
  (the prompt kernel keeps x in bf16, which has float32's smallest step),
  against each code: F = max_j(a_j * V scale) sum_j |V code|.  (A page's scale is at least its
  largest value / 448, so F matters only where the heaviest tokens' own values vanish.)
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import attention_scored_kv_gb300 as kvs
from attention_scored_kv_gb300 import _abi
from oracle import paged as ref

pytestmark = pytest.mark.gpu

DT = {kvs.F32: torch.float32, kvs.BF16: torch.bfloat16}


def make(hq=4, hkv=2, d=32, pages=64, dt=kvs.BF16, kernel=kvs.KERNEL_AUTO, layers=1):
    return kvs.PagedCache(kvs.paged_config_init(num_layers=layers, num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                                                num_pages=pages, in_dtype=dt, kernel=kernel))


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def cpu(t):
    return t.cpu().numpy()


def rand(g, shape, dt, gain=1.0):
    return (torch.randn(shape, generator=g) * gain).to(DT[dt])


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ tables
PLAN_CASES = {
    "one-token": ([0], [1], 4, 8, 1),
    "nothing": ([0], [0], 4, 8, 0),
    "page-edges": ([15, 16, 17, 0, 32, 31], [1, 1, 1, 16, 17, 2], 5, 32, 40),
    "zeros-between": ([5, 0, 7, 0, 0, 9], [0, 3, 0, 0, 0, 20], 4, 16, 23),
    "denied": ([0, 0, 3, 60, 0], [17, 33, 2, 5, 1], 4, 4, 60),
    "rows-cut": ([3, 3], [10, 10], 4, 16, 13),
    "long-row": ([100], [3000], 200, 256, 3001),
    "negative": ([-4, 2], [3, -7], 4, 16, 8),
}


def _plan_inputs(name, seed=5):
    if name in PLAN_CASES:
        return PLAN_CASES[name]
    g = np.random.default_rng(seed)
    n = {"many": 1300, "ragged": 37}[name]
    ctx, new = g.integers(0, 200, n), g.integers(0, 1200 if name == "ragged" else 9, n)
    pages = int((-(-(ctx + new) // 16) - -(-ctx // 16)).sum())
    return ctx, new, 90, pages + (3 if name == "ragged" else -20), int(new.sum()) + 5


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("name", list(PLAN_CASES) + ["ragged", "many"])
def test_plan(name, alias):
    ctx, new, stride, pages, cap = _plan_inputs(name)
    n = len(ctx)
    g = np.random.default_rng(3)
    total = pages + sum(-(-max(int(c), 0) // 16) for c in ctx)
    perm = g.permutation(total)
    table = np.full((n, stride), -1)
    at = 0
    for r in range(n):
        h = -(-max(int(ctx[r]), 0) // 16)
        table[r, :h] = perm[at:at + h]
        at += h
    free = perm[at:]
    cache = make(pages=total)
    want = ref.plan(ctx, new, table, free, len(free), cap)
    t, c, count = i32(table), i32(ctx), i32([len(free)])
    out = count if alias else i32([-9])
    fp = i32(np.concatenate([free, [-1, -1]]))
    p = cache.plan(c, i32(new), t, fp, count, cap, free_count_out=out, kv_len_out=c if alias else None)
    torch.cuda.synchronize()
    assert np.array_equal(cpu(t), want["table"])
    assert np.array_equal(cpu(p.row_start), want["row_start"])
    assert np.array_equal(cpu(p.kv_len), want["kv_len"])
    assert np.array_equal(cpu(p.slots), want["slots"])
    assert np.array_equal(cpu(p.positions), want["positions"])
    assert cpu(out)[0] == want["count"] and cpu(p.denied)[0] == want["denied"]
    if not alias:
        assert np.array_equal(cpu(c), np.asarray(ctx)) and cpu(count)[0] == len(free)
    bad = want["denied"] or sum(max(int(x), 0) for x in new) > cap
    neg = any(int(x) < 0 for x in list(ctx) + list(new))
    assert cache.get_status() == (_abi.ERR_CAPACITY if bad else _abi.ERR_STATE if neg else 0)
    cache.clear_error()
    assert cache.get_status() == 0


def test_slot_map_and_release():
    g = np.random.default_rng(8)
    n, stride = 40, 30
    kv = g.integers(0, stride * 16 + 1, n)
    pages = int((-(-kv // 16)).sum())
    cache = make(pages=pages + 4)
    stack = i32(g.permutation(pages + 4))
    before, count, table = stack.clone(), i32([pages + 4]), torch.full((n, stride), -1, dtype=torch.int32, device="cuda")
    p = cache.plan(i32(np.zeros(n)), i32(kv), table, stack, count, int(kv.sum()))
    assert count.item() == 4
    first = g.integers(0, 20, n) % np.maximum(kv, 1)
    length = np.maximum(kv - first, 0)
    rs, slots, pos = cache.slot_map(i32(length), table, int(length.sum()) + 3, first=i32(first))
    t = cpu(table)
    want_pos = np.concatenate([np.arange(f, f + m) for f, m in zip(first, length)])
    req = np.repeat(np.arange(n), length)
    assert np.array_equal(cpu(rs), np.concatenate([[0], np.cumsum(length)]))
    assert np.array_equal(cpu(pos)[:-3], want_pos)
    assert np.array_equal(cpu(slots), np.concatenate([t[req, want_pos // 16] * 16 + want_pos % 16, [-1] * 3]))
    rs, slots, _ = cache.slot_map(i32(kv), table, int(kv.sum()))
    assert torch.equal(slots, p.slots)
    cache.release(p.kv_len, table, stack, count)
    assert count.item() == pages + 4 and torch.equal(stack, before) and (cpu(table) == -1).all()
    assert cache.get_status() == 0
    cache.release(i32([16]), torch.zeros((1, 1), dtype=torch.int32, device="cuda"), stack, count)     # no room
    assert cache.get_status() == _abi.ERR_CAPACITY and count.item() == pages + 4 and torch.equal(stack, before)


# ------------------------------------------------------------------ append and gather
@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
@pytest.mark.parametrize("hkv,d", [(1, 16), (3, 32), (2, 64), (4, 128)])
def test_append_gather_exact(hkv, d, dt):
    g = torch.Generator().manual_seed(hkv * 100 + d)
    rng = np.random.default_rng(d)
    pages = 40
    cache, orc = make(hq=hkv * 2, hkv=hkv, d=d, pages=pages, dt=dt, layers=2), ref.Pages(pages, hkv, d)
    order = rng.permutation(pages)
    # three requests growing by ragged steps, the values' size growing in some of them
    lens, tables = [0, 0, 0], [order[:12], order[12:24], order[24:36]]
    for step, news in enumerate([(1, 16, 33), (1, 0, 7), (14, 1, 1), (1, 1, 1), (50, 2, 15), (1, 1, 1), (0, 100, 1)]):
        slots = []
        for r, m in enumerate(news):
            p = np.arange(lens[r], lens[r] + m)
            slots += list(tables[r][p // 16] * 16 + p % 16)
            lens[r] += m
        slots += [-1, -1]
        k = rand(g, (len(slots), hkv, d), dt, 4.0 ** (step % 4) / 8)
        v = rand(g, (len(slots), hkv, d), dt, 2.0 ** (-step))
        k[::5, 0] = 0
        cache.append(1, k.cuda(), v.cuda(), i32(slots))
        orc.append(f64(k), f64(v), slots)
        every = np.concatenate([tables[r][np.arange(lens[r]) // 16] * 16 + np.arange(lens[r]) % 16 for r in range(3)])
        every = np.concatenate([every, rng.permutation(every), [-5], every[:3]])
        got = cache.gather(1, i32(every))
        for x, y in zip(got, orc.gather(every)):
            assert np.array_equal(f64(x), y), (step, hkv, d)
    # the whole pool, unwritten slots and the other layer among it
    for layer, o in ((1, orc), (0, ref.Pages(pages, hkv, d))):
        for x, y in zip(cache.gather(layer, i32(np.arange(pages * 16))), o.gather(np.arange(pages * 16))):
            assert np.array_equal(f64(x), y)
    assert cache.get_status() == 0


@pytest.mark.parametrize("rows", [2000, 9000])
def test_append_long(rows):
    """Both ways of dealing rows to warps, runs that do not start at a warp's rows."""
    g = torch.Generator().manual_seed(rows)
    cache, orc = make(hq=2, hkv=1, d=64, pages=700), ref.Pages(700, 1, 64)
    lens = [5, rows - 5 - 37, 37]
    base = np.cumsum([0] + [-(-x // 16) for x in lens])
    slots = np.concatenate([(base[r] * 16 + np.arange(n)) for r, n in enumerate(lens)])
    k, v = rand(g, (rows, 1, 64), kvs.BF16), rand(g, (rows, 1, 64), kvs.BF16)
    cache.append(0, k.cuda(), v.cuda(), i32(slots))
    orc.append(f64(k), f64(v), slots)
    for x, y in zip(cache.gather(0, i32(slots)), orc.gather(slots)):
        assert np.array_equal(f64(x), y)
    assert cache.get_status() == 0


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
def test_append_values_at_the_edges(dt):
    cache, orc = make(hq=1, hkv=1, d=16, pages=4, dt=dt), ref.Pages(4, 1, 16)
    big = torch.finfo(DT[dt]).max
    rows = [[0.0] * 16, [1e-45] * 16, [big] * 16, [float("inf"), float("-inf"), 3.0] + [0.25] * 13,
            [float("nan")] * 8 + [448.0] * 8, [2.0 ** -120, 2.0 ** -110] * 8]
    x = torch.tensor(rows, dtype=torch.float32).to(DT[dt]).view(-1, 1, 16)
    slots = [0, 16, 32, 48, 49, 50]                        # rows of a page are neighbours
    cache.append(0, x.cuda(), x.flip(-1).cuda(), i32(slots))
    orc.append(f64(x), f64(x.flip(-1)), slots)
    for a, b in zip(cache.gather(0, i32(range(64))), orc.gather(np.arange(64))):
        assert np.isfinite(f64(a)).all() and np.array_equal(f64(a), b)
    assert cache.get_status() == _abi.ERR_STATE            # the NaN was reported


def test_slots_out_of_range_are_reported():
    cache = make(hq=1, hkv=1, d=16, pages=2)
    one = torch.ones((3, 1, 16), dtype=torch.bfloat16, device="cuda")
    cache.append(0, one, one, i32([32, 0, 2 ** 31 - 1]))
    assert cache.get_status() == _abi.ERR_STATE
    cache.clear_error()
    k, v = cache.gather(0, i32([0, 1, 32, 2 ** 31 - 1, -2 ** 31]))
    assert cache.get_status() == _abi.ERR_STATE
    assert f64(k)[:, 0, 0].tolist() == [1.0, 0.0, 0.0, 0.0, 0.0]


# ------------------------------------------------------------------ attention
def filled(kv, new, hq, hkv, d, dt, kernel=kvs.KERNEL_AUTO, seed=0, gain=1.0, spare_stride=1):
    """A cache and its oracle holding kv[r] tokens per request in shuffled pages, and queries."""
    g = torch.Generator().manual_seed(seed)
    kv = [int(x) for x in kv]
    n = len(kv)
    blocks = [-(-x // 16) for x in kv]
    pages = sum(blocks) + 3
    stride = max(blocks + [1]) + spare_stride
    perm = np.random.default_rng(seed).permutation(pages)
    table = np.full((n, stride), -7)
    at = 0
    for r in range(n):
        table[r, :blocks[r]] = perm[at:at + blocks[r]]
        at += blocks[r]
    cache, orc = make(hq, hkv, d, pages, dt, kernel), ref.Pages(pages, hkv, d)
    slots = np.concatenate([table[r, np.arange(kv[r]) // 16] * 16 + np.arange(kv[r]) % 16 for r in range(n)] + [np.zeros(0, int)])
    if len(slots):
        rows = len(slots)
        k = rand(g, (rows, hkv, d), dt, gain) * torch.exp(0.5 * torch.randn((1, hkv, d), generator=g)).to(DT[dt])
        v = rand(g, (rows, hkv, d), dt) * torch.exp2(torch.randint(-6, 6, (rows, 1, 1), generator=g).float()).to(DT[dt])
        cache.append(0, k.cuda(), v.cuda(), i32(slots))
        orc.append(f64(k), f64(v), slots)
    q = rand(g, (sum(new), hq, d), dt, 1.5)
    return cache, orc, table, q


def check_out(out, want, d, dt, tensor):
    u = torch.finfo(DT[dt]).eps / 2
    delta = (d + 8) * 2.0 ** -23 * want["reach"] + 2.0 ** -21 * (1 + want["reach"])
    r = 2.0 ** -8 if tensor else 2.0 ** -23
    tol = u * np.abs(want["out"]) + (r + 4 * delta[:, :, None]) * want["spread"] + 1e-30
    if tensor:
        tol += 2.0 ** -23 * want["floor"]
    err = np.abs(f64(out) - want["out"])
    assert np.isfinite(f64(out)).all()
    assert (err <= tol).all(), (err / tol).max()


def check_mass(mass, want, hidden, d):
    delta = (d + 8) * 2.0 ** -23 * want["reach"].max() + 2.0 ** -21 * (1 + want["reach"].max())
    got = f64(mass)
    assert (got[hidden] == -3.0).all()                                  # what is not visible is left as it was
    err = np.abs(got - want["mass"])[~hidden]
    assert (err <= 8 * delta * want["mass"][~hidden] + 1e-30).all(), err.max()


SHAPES = [(8, 2, 16, kvs.F32), (4, 4, 32, kvs.BF16), (32, 4, 128, kvs.BF16), (32, 4, 128, kvs.F32), (12, 4, 64, kvs.BF16),
          (16, 2, 64, kvs.F32), (8, 8, 128, kvs.BF16), (40, 2, 128, kvs.BF16), (64, 1, 64, kvs.BF16)]
DECODE = {"one": [1], "edges": [1, 15, 16, 17, 127, 128, 129, 0, 255, 256, 257], "ragged": [700, 3, 1500, 64, 0, 1023],
          "long": [5000]}


@pytest.mark.parametrize("kernel", [kvs.KERNEL_AUTO, kvs.KERNEL_GENERAL])
@pytest.mark.parametrize("lens", list(DECODE))
@pytest.mark.parametrize("hq,hkv,d,dt", SHAPES)
def test_decode(hq, hkv, d, dt, lens, kernel):
    kv = DECODE[lens]
    if dt == kvs.F32 and kernel == kvs.KERNEL_AUTO:
        pytest.skip("the same kernel")
    n = len(kv)
    cache, orc, table, q = filled(kv, [1] * n, hq, hkv, d, dt, kernel, seed=hq + d)
    tensor = dt == kvs.BF16 and kernel == kvs.KERNEL_AUTO
    t, ln, qd = i32(table), i32(kv), q.cuda()
    want = orc.attend(f64(q), table, kv)
    check_out(cache.attend(0, qd, t, ln), want, d, dt, tensor)
    mass = torch.full(table.shape, -3.0, device="cuda")
    out = cache.attend(0, qd, t, ln, block_mass=mass)
    check_out(out, want, d, dt, tensor)
    hidden = np.arange(table.shape[1])[None] >= -(-np.asarray(kv)[:, None] // 16)
    check_mass(mass, want, hidden, d)
    for window in (1, 17, 200):
        mass.fill_(-3.0)
        want = orc.attend(f64(q), table, kv, window=window)
        check_out(cache.attend(0, qd, t, ln, window=window, block_mass=mass), want, d, dt, tensor)
        first = np.maximum(np.asarray(kv)[:, None] - window, 0) // 16
        check_mass(mass, want, hidden | (np.arange(table.shape[1])[None] < first), d)
    assert cache.get_status() == 0


RAGGED = {
    "few": ([5, 130, 700, 16], [2, 4, 3, 1]),
    "chunks": ([40, 300, 17, 129, 512], [40, 7, 0, 129, 33]),
    "prompt": ([400], [400]),
    "behind": ([1100, 20], [65, 20]),
    "shorter-than-rows": ([3, 0, 20], [5, 2, 1]),
}


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("lens", list(RAGGED))
@pytest.mark.parametrize("hq,hkv,d,dt", SHAPES)
def test_ragged_rows(hq, hkv, d, dt, lens, window):
    kv, new = RAGGED[lens]
    cache, orc, table, q = filled(kv, new, hq, hkv, d, dt, seed=hq + d + window)
    start = np.concatenate([[0], np.cumsum(new)])
    # rows behind the last request's stay as they were
    qd = torch.cat([q.cuda(), torch.full((3, hq, d), float("nan"), dtype=DT[dt], device="cuda")])
    out = torch.full(qd.shape, 9.0, dtype=DT[dt], device="cuda")
    cache.attend(0, qd, i32(table), i32(kv), q_start=i32(start), max_q_len=max(new), window=window, out=out)
    want = orc.attend(f64(q), table, kv, start, window)
    check_out(out[:len(q)], want, d, dt, dt == kvs.BF16 and cache.cfg.kernel != kvs.KERNEL_GENERAL)
    assert (out[len(q):] == 9.0).all()
    assert cache.get_status() == 0


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
def test_few_rows_behind_long_contexts(dt):
    """Work split over the context for rows that are not single tokens."""
    kv, new = [6000, 2500], [4, 9]
    cache, orc, table, q = filled(kv, new, 16, 2, 128, dt, seed=4)
    start = [0, 4, 13]
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=9)
    check_out(out, orc.attend(f64(q), table, kv, start), 128, dt, dt == kvs.BF16)


@pytest.mark.parametrize("hq,hkv,d,dt", [(32, 4, 128, kvs.BF16), (8, 2, 16, kvs.F32)])
def test_large_logits(hq, hkv, d, dt):
    """Logits of several hundred: the maximum moves from page to page, most weights vanish."""
    kv = [900, 333]
    cache, orc, table, q = filled(kv, [1, 1], hq, hkv, d, dt, seed=1, gain=25.0)
    want = orc.attend(f64(q), table, kv)
    check_out(cache.attend(0, q.cuda(), i32(table), i32(kv)), want, d, dt, dt == kvs.BF16)
    kv, new = [600, 90], [70, 30]
    cache, orc, table, q = filled(kv, new, hq, hkv, d, dt, seed=2, gain=25.0)
    want = orc.attend(f64(q), table, kv, [0, 70, 100])
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32([0, 70, 100]), max_q_len=70)
    check_out(out, want, d, dt, dt == kvs.BF16)


def stored(kv, k, v, d, hq, hkv, seed):
    """A cache and its oracle that hold k and v (the requests' tokens one after the other) in shuffled pages."""
    blocks = [-(-x // 16) for x in kv]
    perm = np.random.default_rng(seed).permutation(sum(blocks))
    table, at = np.full((len(kv), max(blocks)), -7), 0
    for r, b in enumerate(blocks):
        table[r, :b] = perm[at:at + b]
        at += b
    slots = np.concatenate([table[r, np.arange(x) // 16] * 16 + np.arange(x) % 16 for r, x in enumerate(kv)])
    cache, orc = make(hq, hkv, d, sum(blocks), kvs.BF16), ref.Pages(sum(blocks), hkv, d)
    cache.append(0, k.cuda(), v.cuda(), i32(slots))
    orc.append(f64(k), f64(v), slots)
    return cache, orc, table


@pytest.mark.parametrize("new", [1, 2, 40, 150])
@pytest.mark.parametrize("d", [64, 128])
def test_logits_that_grow_by_far(d, new):
    """Tokens in either half of a tile whose logits pass all before them by 2^60 to 2^300."""
    g = torch.Generator().manual_seed(d + new)
    kv, hq, hkv = [700, 330], 16, 2
    rows = sum(kv)
    sign = torch.sign(torch.randn((1, 1, d), generator=g))
    size = torch.zeros((rows, 1, 1))
    for j, a in ((3, 0.5), (70, 4), (100, 4.5), (130, 6), (200, 9), (450, 14), (700 + 90, 5), (700 + 180, 10)):
        size[j] = a * (128 / d) ** 0.5
    k = (size * sign + 0.25 * torch.randn((rows, hkv, d), generator=g)).to(torch.bfloat16)
    v = torch.randn((rows, hkv, d), generator=g).to(torch.bfloat16)
    gain = torch.tensor([1.0, 2.0, -1.0, 0.5, -2.0, 0.0, 1.5, 1.0] * 2).view(1, hq, 1)
    q = (gain * sign + 0.1 * torch.randn((2 * new, hq, d), generator=g)).to(torch.bfloat16)
    cache, orc, table = stored(kv, k, v, d, hq, hkv, d)
    start = [0, new, 2 * new]
    want = orc.attend(f64(q), table, kv, start)
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=new)
    check_out(out, want, d, kvs.BF16, True)
    want = orc.attend(f64(q), table, kv, start, window=150)
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=new, window=150)
    check_out(out, want, d, kvs.BF16, True)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("zero", ["first", "last", "odd", "all"])
def test_pages_of_zeros(zero, new):
    """Pages whose values are all 0 have the smallest scale; their tokens keep their weights."""
    g = torch.Generator().manual_seed(new)
    kv, hq, hkv, d = [500, 140], 16, 2, 128
    rows = sum(kv)
    k = torch.randn((rows, hkv, d), generator=g).to(torch.bfloat16)
    v = torch.randn((rows, hkv, d), generator=g)
    pos = torch.cat([torch.arange(x) for x in kv])
    gone = {"first": pos < 128, "last": pos >= 112, "odd": pos // 16 % 2 == 1, "all": pos >= 0}[zero]
    v[gone] = 0
    q = torch.randn((2 * new, hq, d), generator=g).to(torch.bfloat16)
    cache, orc, table = stored(kv, k, v.to(torch.bfloat16), d, hq, hkv, 5)
    start = [0, new, 2 * new]
    want = orc.attend(f64(q), table, kv, start)
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=new)
    check_out(out, want, d, kvs.BF16, True)


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
@pytest.mark.parametrize("new", [[1, 1, 1], [2, 1, 40]])
def test_pages_out_of_range_are_left_out(dt, new):
    kv = [200, 40, 300]
    cache, orc, table, q = filled(kv, new, 16, 2, 128, dt, seed=3)
    table[0, 2], table[0, 5], table[1, :], table[2, 18] = -1, 10 ** 6, 2 ** 31 - 1, cache.cfg.num_pages
    start = np.concatenate([[0], np.cumsum(new)])
    want = orc.attend(f64(q), table, kv, start)
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=max(new))
    check_out(out, want, 128, dt, dt == kvs.BF16)
    assert cache.get_status() == _abi.ERR_STATE
    cache.clear_error()
    if max(new) == 1:
        mass = torch.zeros(table.shape, device="cuda")
        cache.attend(0, q.cuda(), i32(table), i32(kv), block_mass=mass)
        check_mass(mass, want, np.zeros(table.shape, bool), 128)
        assert cache.get_status() == _abi.ERR_STATE


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
def test_lengths_past_what_the_host_said(dt):
    """Lengths beyond the table are cut to it; rows beyond max_q_len are left as they were, and said."""
    kv, new = [64, 64], [6, 2]
    cache, orc, table, q = filled(kv, new, 16, 2, 128, dt, seed=6, spare_stride=0)
    out = torch.full(q.shape, 9.0, dtype=DT[dt], device="cuda")
    cache.attend(0, q.cuda(), i32(table), i32([1000, 64]), q_start=i32([0, 6, 8]), max_q_len=4, out=out)
    assert cache.get_status() == _abi.ERR_CAPACITY
    want = orc.attend(f64(q), table, kv, [0, 6, 8])
    keep = [0, 1, 2, 3, 6, 7]
    check_out(out[keep], {k: v[keep] for k, v in want.items() if k != "mass"}, 128, dt, dt == kvs.BF16)
    assert (out[4:6] == 9.0).all()


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
@pytest.mark.parametrize("n,new", [(700, 1), (600, 5), (1100, 1)])
def test_many_requests(dt, n, new):
    """More requests than the kernels look at in one round, some without rows."""
    rng = np.random.default_rng(n)
    news = rng.integers(0, new + 1, n)
    kv = np.maximum(rng.integers(0, 40, n), news)
    cache, orc, table, q = filled(kv, news, 8, 1, 64, dt, seed=n)
    start = np.concatenate([[0], np.cumsum(news)])
    want = orc.attend(f64(q), table, kv, start)
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=new)
    check_out(out, want, 64, dt, dt == kvs.BF16)
    if new == 1:
        mass = torch.full(table.shape, -3.0, device="cuda")
        out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), block_mass=mass)
        check_out(out, want, 64, dt, dt == kvs.BF16)
        check_mass(mass, want, np.arange(table.shape[1])[None] >= -(-(kv * news)[:, None] // 16), 64)
    assert cache.get_status() == 0


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_queries_that_are_not_finite(dt, new):
    """A query with a NaN or an infinity spoils its own row and head, no other."""
    kv = [90, 200]
    cache, orc, table, q = filled(kv, [new, new], 16, 2, 128, dt, seed=12)
    start = [0, new, 2 * new]
    want = orc.attend(f64(q), table, kv, start)
    bad = q.clone()
    bad[0, 3, 5], bad[new, 9, 127], bad[2 * new - 1, 15, 0] = float("nan"), float("inf"), float("-inf")
    out = cache.attend(0, bad.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=new)
    spoilt = torch.zeros((2 * new, 16), dtype=torch.bool)
    spoilt[0, 3] = spoilt[new, 9] = spoilt[2 * new - 1, 15] = True
    assert out.isnan().any(-1).cpu().equal(spoilt)
    keep = (~spoilt).numpy()
    out[spoilt.cuda()] = 0
    zero = {k: np.where(keep.reshape(keep.shape + (1,) * (v.ndim - 2)), v, 0.0) for k, v in want.items() if k != "mass"}
    check_out(out, zero, 128, dt, dt == kvs.BF16)
    assert cache.get_status() == 0


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
def test_row_starts_that_are_not_sorted(dt):
    """Row starts out of range or falling are reported; rows of the requests that are in order are right."""
    kv, new = [50, 60, 70], [2, 2, 2]
    cache, orc, table, q = filled(kv, new, 16, 2, 128, dt, seed=13)
    want = orc.attend(f64(q), table, kv, [0, 2, 4, 6])
    for start, good in (([0, 2, 1, 1], [0, 1]), ([-3, 2, 4, 6], [2, 3, 4, 5]), ([0, 2, 4, 9], [0, 1, 2, 3])):
        for most in (2, 9):
            out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=most)
            if dt == kvs.BF16:              # the other path looks rows up by their starts, which need an order
                check_out(out[good], {k: v[good] for k, v in want.items() if k != "mass"}, 128, dt, True)
            assert cache.get_status() == _abi.ERR_CAPACITY
            cache.clear_error()


def test_windows_past_every_length():
    kv, new = [300, 20], [1, 1]
    cache, orc, table, q = filled(kv, new, 8, 1, 64, kvs.BF16, seed=14)
    plain = cache.attend(0, q.cuda(), i32(table), i32(kv))
    for window in (300, 10 ** 6, 2 ** 31 - 1):
        assert torch.equal(cache.attend(0, q.cuda(), i32(table), i32(kv), window=window), plain)
    rag = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32([0, 1, 2]), max_q_len=50)
    assert torch.equal(cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32([0, 1, 2]), max_q_len=50, window=2 ** 31 - 1), rag)


# ------------------------------------------------------------------ a run of them together
def step_graph(cache, st, layers, cap, q_len):
    """One step as a program would capture it: everything from static tensors."""
    p = cache.plan(st["len"], st["new"], st["table"], st["free"], st["count"], cap, kv_len_out=st["len"])
    outs = []
    for layer in range(layers):
        cache.append(layer, st["k"][layer], st["v"][layer], p.slots)
        if q_len == 1:
            outs.append(cache.attend(layer, st["q"][layer], st["table"], st["len"], block_mass=st["mass"]))
        else:
            outs.append(cache.attend(layer, st["q"][layer], st["table"], st["len"], q_start=p.row_start, max_q_len=q_len))
    return p, outs


@pytest.mark.parametrize("q_len", [1, 3])
def test_steps_captured_and_replayed(q_len):
    """Plan, append and attend of two layers in one graph, replayed while requests grow: the
    same bytes as eager calls, and the oracle's outputs; then the pages are released."""
    hq, hkv, d, n, layers, steps, stride = 16, 2, 128, 5, 2, 12, 6
    pages, cap = n * stride + 2, n * q_len
    g = torch.Generator().manual_seed(q_len)
    ks, vs, qs = ([rand(g, (layers, cap, h, d), kvs.BF16).cuda() for _ in range(steps)] for h in (hkv, hkv, hq))
    news = [np.random.default_rng(s).integers(q_len - 1 if q_len > 1 else 1, q_len + 1, n) for s in range(steps)]
    start = np.array([0, 30, 15, 16, 1])
    perm = np.random.default_rng(0).permutation(pages)

    def fresh():
        cache = make(hq, hkv, d, pages, layers=layers)
        st = {"len": i32(np.zeros(n)), "new": i32(start), "free": i32(perm), "count": i32([pages]),
              "table": torch.full((n, stride), -1, dtype=torch.int32, device="cuda"),
              "mass": torch.zeros((n, stride), device="cuda"),
              "k": torch.zeros_like(ks[0]), "v": torch.zeros_like(vs[0]), "q": torch.zeros_like(qs[0])}
        rows = int(start.sum())
        p = cache.plan(st["len"], st["new"], st["table"], st["free"], st["count"], rows, kv_len_out=st["len"])
        g2 = torch.Generator().manual_seed(99)
        k0, v0 = rand(g2, (rows, hkv, d), kvs.BF16), rand(g2, (rows, hkv, d), kvs.BF16)
        for layer in range(layers):
            cache.append(layer, k0.cuda(), v0.cuda(), p.slots)
        return cache, st, k0, v0, p

    def feed(st, s):
        st["new"].copy_(i32(news[s]))
        for name, src in (("k", ks), ("v", vs), ("q", qs)):
            st[name].copy_(src[s])

    eager, st_e, k0, v0, p0 = fresh()
    graphed, st_g, _, _, _ = fresh()
    orcs = [ref.Pages(pages, hkv, d) for _ in range(layers)]
    for o in orcs:
        o.append(f64(k0), f64(v0), cpu(p0.slots))
    # warm-up on a side stream with rows that store nothing, then capture
    zero = i32(np.zeros(n))
    st_g["new"].copy_(zero)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step_graph(graphed, st_g, layers, cap, q_len)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p_g, outs_g = step_graph(graphed, st_g, layers, cap, q_len)
    for s in range(steps):
        feed(st_e, s)
        feed(st_g, s)
        p_e, outs_e = step_graph(eager, st_e, layers, cap, q_len)
        graph.replay()
        torch.cuda.synchronize()
        rows = int(news[s].sum())
        assert torch.equal(st_e["table"], st_g["table"]) and torch.equal(st_e["len"], st_g["len"])
        assert torch.equal(p_e.slots, p_g.slots)
        for layer in range(layers):
            assert torch.equal(outs_e[layer][:rows], outs_g[layer][:rows])
            orcs[layer].append(f64(ks[s][layer]), f64(vs[s][layer]), cpu(p_e.slots))
            want = orcs[layer].attend(f64(qs[s][layer])[:rows], cpu(st_e["table"]), cpu(st_e["len"]), cpu(p_e.row_start))
            check_out(outs_e[layer][:rows], want, d, kvs.BF16, True)
        if q_len == 1:
            assert torch.equal(st_e["mass"], st_g["mass"])
    for cache, st in ((eager, st_e), (graphed, st_g)):
        assert cache.get_status() == 0, cache.last_error()
        cache.release(st["len"], st["table"], st["free"], st["count"])
        assert st["count"].item() == pages and sorted(cpu(st["free"])) == list(range(pages))


def test_two_streams_at_once():
    """Two attends of one cache on two streams, and calls on a stream that is not current."""
    kv = [2000, 1700, 900]
    cache, orc, table, q = filled(kv, [1, 1, 1], 32, 4, 128, kvs.BF16, seed=9)
    t, ln, qd = i32(table), i32(kv), q.cuda()
    want = cache.attend(0, qd, t, ln)
    want2 = cache.attend(0, qd, t, ln, window=100)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((cache.attend(0, qd, t, ln, stream=a), cache.attend(0, qd, t, ln, window=100, stream=b)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want) and torch.equal(y, want2)
    check_out(want, orc.attend(f64(q), table, kv), 128, kvs.BF16, True)


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
def test_both_ways_of_calling(dt):
    """The extension and the methods' own path give the same bytes and refuse the same calls."""
    kv, new = [100, 37, 250], [1, 1, 1]
    cache, _, table, q = filled(kv, new, 8, 2, 64, dt, seed=20)
    t, ln, qd = i32(table), i32(kv), q.cuda()
    g = torch.Generator().manual_seed(1)
    k, v = rand(g, (20, 2, 64), dt).cuda(), rand(g, (20, 2, 64), dt).cuda()
    slots = i32(16 * int(table[0, 0]) + np.arange(20) % 16)[:16]
    k, v = k[:16], v[:16]
    results = []
    for fast in (cache._fast, None):
        cache._fast = fast
        free, count, tab = i32(np.arange(30)), i32([30]), torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
        p = cache.plan(i32([0, 5, 16]), i32([17, 3, 0]), tab, free, count, 23)
        cache.append(0, k, v, slots)
        mass = torch.zeros(t.shape, device="cuda")
        results.append([tab, count, *p, *cache.gather(0, slots), cache.attend(0, qd, t, ln, block_mass=mass), mass,
                        cache.attend(0, qd, t, ln, q_start=i32([0, 1, 2, 3]), max_q_len=50, window=33)])
        for call in (lambda: cache.append(0, k, v, slots.long()), lambda: cache.gather(0, slots.cpu()),
                     lambda: cache.attend(0, qd.double(), t, ln), lambda: cache.plan(ln, ln, t.float(), ln, count, 3)):
            with pytest.raises(TypeError):
                call()
        for call in (lambda: cache.append(3, k, v, slots), lambda: cache.gather(-1, slots), lambda: cache.attend(1, qd, t, ln),
                     lambda: cache.attend(0, qd, t, ln, max_q_len=2), lambda: cache.plan(ln, ln, t, ln, count, (1 << 30) + 4)):
            with pytest.raises((kvs.KVSError, torch.OutOfMemoryError)):
                call()
        cache.clear_error()
    for a, b in zip(*results):
        assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)
    class Own(torch.Tensor):
        pass
    out = cache.attend(0, qd.as_subclass(Own), t, ln)
    assert torch.equal(out, results[0][-3])


def test_two_graphs_at_once():
    """Two captured graphs over one cache, replayed on two streams: each has scratch of its own."""
    kv, new = [1500, 700, 300], [1, 1, 60]
    cache, orc, table, q = filled(kv, new, 16, 2, 128, kvs.BF16, seed=21)
    t, ln, qd, st = i32(table), i32(kv), q.cuda(), i32([0, 1, 2, 62])
    calls = [lambda: cache.attend(0, qd, t, ln, q_start=st, max_q_len=60),
             lambda: cache.attend(0, qd[:3], t, ln, window=900),
             lambda: cache.attend(0, qd, t, ln, q_start=st, max_q_len=60, window=50)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append([c() for _ in range(6)])
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, many in zip(want, outs):
        for o in many:
            assert torch.equal(o, w)
    assert cache.get_status() == 0


@pytest.mark.parametrize("dt", [kvs.BF16, kvs.F32])
def test_pages_beyond_32_bits(dt):
    """A pool whose codes pass 4 GB in each of K and V, used at its ends."""
    pages, hkv, d = 600_000, 4, 128
    cache, orc = make(16, hkv, d, pages, dt), ref.Pages(40, hkv, d)
    ids = np.concatenate([np.arange(20), pages - 20 + np.arange(20)])[np.random.default_rng(0).permutation(40)]
    table, small = ids.reshape(2, 20), np.arange(40).reshape(2, 20)
    kv, g = [317, 290], torch.Generator().manual_seed(3)
    slots, own = (np.concatenate([t[r, np.arange(n) // 16] * 16 + np.arange(n) % 16 for r, n in enumerate(kv)]) for t in (table, small))
    k, v, q = rand(g, (sum(kv), hkv, d), dt), rand(g, (sum(kv), hkv, d), dt), rand(g, (92, 16, d), dt)
    cache.append(0, k.cuda(), v.cuda(), i32(slots))
    orc.append(f64(k), f64(v), own)
    for x, y in zip(cache.gather(0, i32(slots)), orc.gather(own)):
        assert np.array_equal(f64(x), y)
    for n in ([1, 1], [2, 90]):
        start = [0, n[0], n[0] + n[1]]
        out = cache.attend(0, q[:sum(n)].cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=max(n))
        check_out(out, orc.attend(f64(q[:sum(n)]), small, kv, start), d, dt, dt == kvs.BF16)
    assert cache.get_status() == 0


# ------------------------------------------------------------------ refusals (all on the host, before any launch)
def test_refusals():
    cache, orc, table, q = filled([40, 20], [1, 1], 4, 2, 32, kvs.BF16)
    t, ln, qd = i32(table), i32([40, 20]), q.cuda()
    one = torch.zeros((3, 2, 32), dtype=torch.bfloat16, device="cuda")
    s3 = i32([0, 1, 2])

    def refused(status, f, *a, **kw):
        with pytest.raises(kvs.KVSError) as e:
            f(*a, **kw)
        assert e.value.status == status and cache.last_error()

    inv, uns, cap = _abi.ERR_INVALID_ARGUMENT, _abi.ERR_UNSUPPORTED, _abi.ERR_CAPACITY
    refused(inv, cache.append, 1, one, one, s3)
    refused(inv, cache.append, -1, one, one, s3)
    refused(inv, cache.gather, 1, s3)
    refused(inv, cache.attend, 2, qd, t, ln)
    refused(inv, cache.attend, 0, qd, t, ln, window=-1)
    refused(inv, cache.attend, 0, qd, t, ln, max_q_len=0, q_start=i32([0, 1, 2]), scratch=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    refused(inv, cache.attend, 0, torch.cat([qd, qd]), t, ln)                       # rows without q_start
    refused(inv, cache.attend, 0, qd, t, ln, out=qd)
    refused(uns, cache.attend, 0, qd, t, ln, q_start=i32([0, 1, 2]), max_q_len=2, block_mass=torch.zeros(t.shape, device="cuda"),
            scratch=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    refused(cap, cache.attend, 0, qd, t, ln, block_mass=torch.zeros(t.shape, device="cuda"),
            scratch=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    refused(inv, cache.attend, 0, qd, t, ln, scratch=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")[8:])
    odd = torch.zeros(3 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(3, 2, 32)
    refused(inv, cache.append, 0, odd, one, s3)
    refused(inv, cache.gather, 0, s3, k_out=odd, v_out=one)
    for call in (lambda: cache.append(0, one.float(), one, s3), lambda: cache.append(0, one.cpu(), one, s3),
                 lambda: cache.attend(0, qd.float(), t, ln), lambda: cache.attend(0, qd, t.long(), ln),
                 lambda: cache.attend(0, qd, t, ln, block_mass=torch.zeros(t.shape, dtype=torch.float64, device="cuda")),
                 lambda: cache.plan(ln, ln, t, ln.cpu(), i32([1]), 4)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: cache.append(0, one[:2], one[:2], s3), lambda: cache.append(0, one, one, s3[::2]),
                 lambda: cache.append(0, one.transpose(0, 2), one, s3), lambda: cache.attend(0, qd, t, ln[:1]),
                 lambda: cache.attend(0, qd, t[:, ::2], ln), lambda: cache.attend(0, qd, t, ln, q_start=i32([0, 1])),
                 lambda: cache.plan(ln, ln, t, ln, ln, 4), lambda: cache.plan(ln, ln, t, ln, i32([1]), -1)):
        with pytest.raises(ValueError):
            call()
    assert cache.get_status() == 0
    # calls with no rows do nothing
    cache.append(0, one[:0], one[:0], s3[:0])
    assert cache.gather(0, s3[:0])[0].shape == (0, 2, 32)
    assert cache.attend(0, qd[:0], t, ln, q_start=i32([0, 0, 0])).shape == (0, 4, 32)
    wide = torch.zeros((1, (1 << 22) + 1), dtype=torch.int32, device="cuda")
    refused(inv, cache.attend, 0, qd[:1], wide, ln[:1], scratch=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kvs.KVSError):
        make(d=96)
    with pytest.raises(kvs.KVSError):
        make(d=16, kernel=kvs.KERNEL_TENSOR)
    with pytest.raises(kvs.KVSError):
        make(dt=kvs.F32, d=128, kernel=kvs.KERNEL_TENSOR)


def test_debug_build():
    """The same operators with the checked build, in a process of its own."""
    env = dict(os.environ, KVS_LIB_VARIANT="debug", KVS_NVTX="1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", os.path.abspath(__file__), "-k",
                        "captured or (test_decode and edges and 128) or out_of_range"], cwd=root, env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:]
