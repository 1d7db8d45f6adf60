"""Whole numbers that do not fit the paged calls' 32-bit arguments (no GPU needed)."""
import ctypes

import pytest

import attention_scored_kv_gb300 as kvs
from attention_scored_kv_gb300 import _abi
from tests.test_abi_host import built_library  # noqa: F401  (builds the library once)

CALLS = {                                # the calls' arguments, 0 at every 32-bit one
    "plan": [None, 0, None, None, None, 0, None, 0, *[None] * 6, 0, None, None],
    "slot_map": [None, 0, None, None, None, 0, None, None, None, 0, None],
    "release": [None, 0, None, None, 0, None, 0, None, None],
    "append": [None, 0, 0, None, None, None, None],
    "gather": [None, 0, 0, None, None, None, None],
    "attend": [None, 0, 0, None, 0, None, None, 0, 0, 0, *[None] * 4, 0, None],
    "attend_scratch_bytes": [None, 0, 0, 0, 0, 0],
}


@pytest.mark.parametrize("value", [2 ** 32, 2 ** 32 + 5, 2 ** 31, -2 ** 31 - 1, -2 ** 32, 2 ** 70])
@pytest.mark.parametrize("name", list(CALLS))
def test_what_does_not_fit_is_refused(name, value):
    """Cut to its low bits, 2^32 would be layer 0 and 2^32 + 5 a window of 5."""
    fn = getattr(kvs.lib(), "kvs_paged_" + name)
    fn(*CALLS[name])                                       # a null handle: refused by status
    for i, (x, t) in enumerate(zip(CALLS[name], fn.argtypes)):
        if t is ctypes.c_size_t or x is None:
            continue
        with pytest.raises((ctypes.ArgumentError, OverflowError)):
            fn(*CALLS[name][:i], value, *CALLS[name][i + 1:])


@pytest.mark.parametrize("field", ["num_layers", "num_pages", "head_dim", "kernel"])
def test_config_fields(field):
    with pytest.raises(ValueError):
        kvs.paged_config_init(**{field: 2 ** 32 + 16})
    assert getattr(kvs.paged_config_init(**{field: 16}), field) == 16
    assert _abi.int32(2 ** 31 - 1) == 2 ** 31 - 1
