"""The package without the things that only the paged cache's speed needs (no GPU needed)."""
import os
import subprocess
import sys

from tests.test_abi_host import built_library  # noqa: F401  (builds the library once)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def child(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_import_with_a_torch_that_has_no_cuda():
    """Its torch._C lacks the stream functions; configs and sizes are host calls."""
    out = child("import torch\n"
                "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
                "import attention_scored_kv_gb300 as kvs\n"
                "c = kvs.paged_config_init(num_layers=1, num_q_heads=8, num_kv_heads=2, head_dim=64, num_pages=4)\n"
                "print(kvs.paged_workspace_bytes(c) > 0, kvs.workspace_bytes(kvs.config_init()) >= 0)\n")
    assert out.split() == ["True", "True"]
