"""Host-side checks of the paged cache's C ABI and binding (no GPU needed)."""
import ctypes

import pytest
import torch

import attention_scored_kv_gb300 as kvs
from attention_scored_kv_gb300 import _abi, paged
from tests.test_abi_host import built_library  # noqa: F401  (builds the library once)


def cfg(**kw):
    base = dict(num_layers=10, num_q_heads=32, num_kv_heads=4, head_dim=128, num_pages=1000)
    base.update(kw)
    return kvs.paged_config_init(**base)


def test_defaults():
    c = kvs.paged_config_init()
    assert (c.block_tokens, c.in_dtype, c.kernel, c.num_layers) == (16, kvs.BF16, kvs.KERNEL_AUTO, 0)


@pytest.mark.parametrize("field,value,status", [
    ("num_layers", 0, _abi.ERR_INVALID_ARGUMENT), ("num_q_heads", 30, _abi.ERR_INVALID_ARGUMENT),
    ("num_kv_heads", 0, _abi.ERR_INVALID_ARGUMENT), ("num_q_heads", 4 * 65, _abi.ERR_UNSUPPORTED),
    ("head_dim", 96, _abi.ERR_UNSUPPORTED), ("head_dim", 256, _abi.ERR_UNSUPPORTED),
    ("num_pages", 0, _abi.ERR_INVALID_ARGUMENT), ("num_pages", 1 << 27, _abi.ERR_UNSUPPORTED),
    ("block_tokens", 32, _abi.ERR_UNSUPPORTED), ("in_dtype", kvs.E4M3, _abi.ERR_INVALID_ARGUMENT),
    ("kernel", 3, _abi.ERR_INVALID_ARGUMENT),
])
def test_bad_configs_are_refused(field, value, status):
    c = cfg(**{field: value})
    st, msg = kvs.validate_paged_config(c)
    assert st == status and msg
    assert kvs.paged_workspace_bytes(c) == 0
    with pytest.raises(kvs.KVSError):
        kvs.PagedCache(c)


def test_reserved_fields_must_be_zero():
    c = cfg()
    c.reserved[5] = 1
    assert kvs.validate_paged_config(c)[0] == _abi.ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("hkv,d,pages,layers", [(4, 128, 1000, 10), (1, 16, 1, 1), (3, 64, 77, 2)])
def test_workspace_bytes(hkv, d, pages, layers):
    n = kvs.paged_workspace_bytes(cfg(num_q_heads=hkv, num_kv_heads=hkv, head_dim=d, num_pages=pages, num_layers=layers))
    need = layers * pages * hkv * (2 * 16 * d + 8)
    assert need <= n <= need + 4 * 256 + 256 and n % 256 == 0


def test_null_handles_are_refused():
    lib = kvs.lib()
    nul = ctypes.c_void_p()
    assert lib.kvs_paged_destroy(nul) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_get_status(nul, None) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_clear_error(nul, None) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_append(nul, 0, 1, None, None, None, None) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_gather(nul, 0, 1, None, None, None, None) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_plan(nul, 1, *[None] * 3, 1, None, 0, *[None] * 6, 0, None, None) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_slot_map(nul, 1, *[None] * 3, 1, *[None] * 3, 0, None) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_release(nul, 1, None, None, 1, None, 0, None, None) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_attend(nul, 0, 1, None, 1, None, None, 1, 1, 0, *[None] * 4, 0, None) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_attend_scratch_bytes(nul, 1, 1, 1, 1, 0) == 0
    assert lib.kvs_paged_last_error(nul) == b""
    out = ctypes.c_void_p()
    c = cfg()
    assert lib.kvs_paged_create(ctypes.byref(c), None, 1 << 30, None, ctypes.byref(out)) == _abi.ERR_INVALID_ARGUMENT
    assert lib.kvs_paged_create(ctypes.byref(c), 256, 256, None, ctypes.byref(out)) == _abi.ERR_CAPACITY
    assert lib.kvs_paged_create(ctypes.byref(c), 264, 1 << 40, None, ctypes.byref(out)) == _abi.ERR_INVALID_ARGUMENT
    assert not out.value


def test_binding_refuses_host_tensors():
    cache = object.__new__(kvs.PagedCache)
    cache.cfg, cache.device, cache.in_dtype = cfg(), torch.device("cuda", 0), torch.bfloat16
    cache._index, cache._row, cache._qrow = 0, (4, 128), (32, 128)
    ints = torch.zeros(4, dtype=torch.int32)
    kv = torch.zeros((4, 4, 128), dtype=torch.bfloat16)
    for call in (lambda: cache.append(0, kv, kv, ints), lambda: cache.gather(0, ints),
                 lambda: cache.attend(0, kv, ints.view(2, 2), ints), lambda: cache.plan(ints, ints, ints, ints, ints, 1),
                 lambda: cache.release(ints, ints, ints, ints), lambda: cache.slot_map(ints, ints, 1)):
        with pytest.raises(TypeError):
            call()


def test_plan_tuple_names():
    p = paged.PagedPlan(1, 2, 3, 4, 5)
    assert p.q_start == p.row_start == 1 and p.kv_len == 2 and p.denied == 5
