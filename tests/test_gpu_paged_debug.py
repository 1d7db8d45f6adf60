"""The checked build (libkvs_debug.so) on the paged cache: scratch that starts as NaN, bounds
checks of what comes from device memory.  In processes of their own, as a library is loaded once."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

POISON = r'''
import numpy as np, torch
import attention_scored_kv_gb300 as kvs
from tests.test_gpu_paged import filled, i32, check_out
assert bool(kvs.lib().kvs_build_info() & 1) == %d
for kv, new in (([2000, 1700, 900], [1, 1, 1]), ([700, 3000], [60, 9])):
    cache, orc, table, q = filled(kv, new, 32, 4, 128, kvs.BF16, seed=1)
    start = np.concatenate([[0], np.cumsum(new)])
    n = cache.attend_scratch_bytes(len(kv), table.shape[1], len(q), max(new))
    scratch = torch.zeros((n + 4096,), dtype=torch.uint8, device="cuda")
    out = cache.attend(0, q.cuda(), i32(table), i32(kv), q_start=i32(start), max_q_len=max(new), scratch=scratch)
    check_out(out, orc.attend(q.double().numpy(), table, kv, start), 128, kvs.BF16, True)
    words = scratch[:n].view(torch.int32)
    print(int((words == -1).sum()) > 0, int(scratch[n:].sum()) == 0, cache.get_status())
'''


@pytest.mark.parametrize("variant", ["debug", ""])
def test_scratch_starts_as_nan_in_the_checked_build_only(variant):
    env = dict(os.environ, KVS_LIB_VARIANT=variant)
    r = subprocess.run([sys.executable, "-c", POISON % (variant == "debug")], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert r.stdout.splitlines() == ["%s True 0" % (variant == "debug")] * 2


def test_the_paged_tests_in_the_checked_build():
    """Cuts over many requests, all kernels, masses, prompts, unsorted starts and captured steps: no read of
    scratch that was not written, no index out of range."""
    env = dict(os.environ, KVS_LIB_VARIANT="debug")
    files = [os.path.join(ROOT, "tests", f) for f in ("test_gpu_paged.py", "test_gpu_paged_weights.py", "test_gpu_paged_tables.py")]
    pick = ("ragged_rows or test_decode or many_requests or not_sorted or host_said or long_contexts or captured or two_graphs or "
            "out_of_range or append or release or (masses and 600) or (sinks_without and 5000)")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", *files, "-k", pick], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "passed" in r.stdout, r.stdout[-3000:]
