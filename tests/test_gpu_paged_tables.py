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
