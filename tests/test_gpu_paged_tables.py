"""Page tables at the ends of their ranges."""
import numpy as np
import pytest
import torch

import attention_scored_kv_gb300 as kvs
from attention_scored_kv_gb300 import _abi
from oracle import paged as ref
from tests.test_gpu_paged import cpu, i32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("alias", [False, True])
def test_plan_that_wants_more_pages_than_32_bits_count(alias):
    """512 requests that want 2^22 pages each behind one that gets its page, and one behind them that wants none."""
    n, stride, cap = 514, 1 << 22, 40
    cache = make(pages=9)
    table = torch.empty((n, stride), dtype=torch.int32, device="cuda")            # 8.6 GB
    table[0, :3], table[n - 1, :3] = i32([-5, -6, -7]), i32([8, -6, -7])
    new = np.full(n, 1 << 26)
    new[0], new[n - 1] = 16, 4
    ctx = np.zeros(n, int)
    ctx[n - 1] = 8
    c, count = i32(ctx), i32([5])
    out = count if alias else i32([-1])
    p = cache.plan(c, i32(new), table, i32([7, 1, 2, 3, 4]), count, cap, free_count_out=out, kv_len_out=c if alias else None)
    torch.cuda.synchronize()
    assert cpu(table[0, :3]).tolist() == [4, -6, -7] and cpu(table[n - 1, :3]).tolist() == [8, -6, -7]
    assert cpu(p.denied)[0] == 512 and cpu(out)[0] == 4
    assert cpu(p.kv_len).tolist() == [16] + [0] * 512 + [12]
    assert cpu(p.slots).tolist() == [64 + i for i in range(16)] + [-1] * (cap - 16)
    assert cpu(p.positions).tolist() == list(range(16)) + list(range(cap - 16))
    assert cpu(p.row_start)[[0, 1, 2]].tolist() == [0, 16, 16 + (1 << 26)]
    assert cache.get_status() == _abi.ERR_CAPACITY


def test_calls_with_more_work_than_a_cta_counts_are_refused():
    """By the sizes alone, before any array is looked at."""
    cache = make(hq=64, hkv=8, d=128, pages=2)
    lib = kvs.lib()
    for n, stride, rows, most in ((1 << 20, 1 << 22, 1 << 20, 1), (1, 1 << 22, 1 << 28, 1 << 28)):
        assert lib.kvs_paged_attend_scratch_bytes(cache._ctx, n, stride, rows, most, 0) == 0
        st = lib.kvs_paged_attend(cache._ctx, 0, n, None, stride, None, 256, rows, most, 0, *[None] * 4, 0, None)
        assert st == _abi.ERR_UNSUPPORTED and "too much for one call" in cache.last_error()
    assert lib.kvs_paged_attend_scratch_bytes(cache._ctx, 1024, 8192, 1024, 1, 0) > 0


def released(kv, table, stack, count, num_pages):
    """kvs_paged_release in plain Python: (stack, count, table)."""
    stack, table, order = list(stack), np.array(table), []
    for r, x in enumerate(kv):
        for b in range(min(-(-max(int(x), 0) // 16), table.shape[1])):
            if 0 <= table[r, b] < num_pages:
                order.append(table[r, b])
            table[r, b] = -1
    for page in reversed(order):
        if count < len(stack):
            stack[count] = page
            count += 1
    return stack, count, table


@pytest.mark.parametrize("n,stride,room", [(1, 1, 0), (1, 1, 9), (3, 40, 0), (5, 3000, 100), (256, 9, 3), (257, 40, 0), (900, 30, -500)])
@pytest.mark.parametrize("bad", [0.0, 0.2, 1.0])
def test_release_leaves_out_what_is_not_a_page(n, stride, room, bad):
    """A later plan gets pages only; their order is the reverse of the one that they were taken in."""
    rng = np.random.default_rng(n + stride)
    kv = rng.integers(-3, stride * 16 + 40, n)
    blocks = np.minimum(-(-np.maximum(kv, 0) // 16), stride)
    pages = int(blocks.sum()) + 3
    table = np.full((n, stride), -9)
    perm, at = rng.permutation(pages), 0
    for r, b in enumerate(blocks):
        table[r, :b] = perm[at:at + b]
        at += b
    spoilt = (rng.random((n, stride)) < bad) & (np.arange(stride)[None] < blocks[:, None])
    table[spoilt] = rng.choice([-1, pages, 2 ** 31 - 1, -2 ** 31], int(spoilt.sum()))
    stack = np.concatenate([perm[at:], np.full(max(pages - 3 + room, 0), -7)])
    cache = make(hq=1, hkv=1, d=16, pages=pages)
    t, s, c = i32(table), i32(stack), i32([3])
    cache.release(i32(kv), t, s, c)
    want_s, want_c, want_t = released(kv, table, stack, 3, pages)
    assert cpu(c)[0] == want_c and cpu(s).tolist() == list(want_s) and np.array_equal(cpu(t), want_t)
    got = cpu(s)[:want_c]
    assert ((got >= 0) & (got < pages)).all() and len(set(got.tolist())) == want_c
    full = len(blocks) and int((table[np.arange(stride)[None] < blocks[:, None]] >= 0).sum()) > len(stack) - 3
    st = cache.get_status()
    assert st in ((_abi.ERR_STATE, _abi.ERR_CAPACITY) if spoilt.any() or full else (0,))


def test_a_plan_whose_outputs_fail_takes_its_pages_once():
    """The extension's views fail (as under a dispatch mode that refuses them): the method makes the call, once."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class NoStrided(TorchDispatchMode):
        seen = 0

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if "as_strided" in str(func):
                NoStrided.seen += 1
                raise RuntimeError("refused")
            return func(*args, **(kwargs or {}))

    cache = make(pages=20)
    table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
    ctx, new, free, count = i32([0, 0]), i32([20, 5]), i32(np.arange(20)), i32([20])
    with NoStrided():
        p = cache.plan(ctx, new, table, free, count, 25)
    assert NoStrided.seen == 1
    assert cpu(count)[0] == 17 and cpu(table)[:, :2].tolist() == [[19, 18], [17, -1]]
    assert cpu(p.slots)[:3].tolist() == [304, 305, 306] and cpu(p.kv_len).tolist() == [20, 5]
