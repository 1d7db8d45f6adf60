"""Memory of the paged cache's calls on a stream that is not the current one."""
import numpy as np
import pytest
import torch

import attention_scored_kv_gb300 as kvs
from tests.test_gpu_paged import filled, i32

pytestmark = pytest.mark.gpu


def storages(x):
    return {t.untyped_storage().data_ptr(): t.untyped_storage().nbytes()
            for t in (x if isinstance(x, (tuple, list)) else (x,)) if t.numel()}


@pytest.mark.parametrize("name", ["plan", "slot_map", "gather", "attend"])
def test_memory_in_use_on_the_current_stream_is_not_taken(name):
    """A tensor that was just freed while the current stream still reads it keeps its bytes."""
    n, rows = 64, 60000
    cache, _, table, q = filled([300] * n, [1] * n, 32, 4, 128, kvs.BF16, seed=3)
    t, ln, qd, slots = i32(table), i32([300] * n), q.cuda(), i32(np.zeros(rows))
    free, count = i32(np.arange(5)), i32([5])
    calls = {
        "plan": lambda s: cache.plan(ln, i32(np.zeros(n)), t, free, count, rows, stream=s),
        "slot_map": lambda s: cache.slot_map(ln, t, rows, stream=s),
        "gather": lambda s: cache.gather(0, slots, stream=s),
        "attend": lambda s: cache.attend(0, qd, t, ln, stream=s),
    }
    want = [x.clone() for x in (lambda r: r if isinstance(r, tuple) else (r,))(calls[name](None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks of the sizes that the call will ask for, written late on the current stream
    sizes = [x.untyped_storage().nbytes() for x in want]
    sizes += [cache.attend_scratch_bytes(n, table.shape[1], n)] if name == "attend" else []
    held = [torch.zeros(s, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(2)]
    at = {h.data_ptr() for h in held}
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                          # about 10 ms
    late = [h + 1 for h in held]
    del held
    got = calls[name](side)
    assert not at & set(storages(got))
    torch.cuda.synchronize()
    assert all((x == 1).all() for x in late)
    for x, y in zip(got if isinstance(got, tuple) else (got,), want):
        assert torch.equal(x, y)
    assert cache.get_status() == 0


def test_a_cache_made_and_used_on_side_streams():
    """The workspace is zeroed, used and given back with work on several streams."""
    want = None
    for _ in range(3):
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        cache = kvs.PagedCache(kvs.paged_config_init(num_layers=1, num_q_heads=8, num_kv_heads=2, head_dim=64, num_pages=40), stream=a)
        g = torch.Generator().manual_seed(1)
        k, v = (torch.randn((100, 2, 64), generator=g).bfloat16().cuda() for _ in range(2))
        q, slots = torch.randn((1, 8, 64), generator=g).bfloat16().cuda(), i32(np.arange(100))
        table, ln = i32(np.arange(7)[None]), i32([100])
        torch.cuda.synchronize()
        cache.append(0, k, v, slots, stream=a)
        b.wait_stream(a)
        out = cache.attend(0, q, table, ln, stream=b)
        with torch.cuda.stream(b):
            out2 = cache.attend(0, q, table, ln)
        del cache                                          # its memory is not reused before b has run
        junk = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(out, out2) and torch.isfinite(out).all() and junk.numel()
        want = out if want is None else want
        assert torch.equal(out, want)
