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


def test_build_without_a_host_compiler(monkeypatch, capsys):
    """libkvs.so needs nvcc only; the extension is left out, and said to be."""
    from attention_scored_kv_gb300 import build
    monkeypatch.setattr(build.shutil, "which", lambda name, real=build.shutil.which: None if name == "g++" else real(name))
    assert build._build_call() is None
    assert "g++" in capsys.readouterr().err
    monkeypatch.undo()
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build._build_call() is None
    assert "torch" in capsys.readouterr().err


def test_a_cache_without_the_extension():
    """Missing, or built for another torch: a warning, and every method's own path."""
    out = child("import os, tempfile, warnings\n"
                "import attention_scored_kv_gb300 as kvs\n"
                "from attention_scored_kv_gb300 import _abi, paged\n"
                "kvs.lib()\n"
                "for content in (None, b'not a library'):\n"
                "    d = tempfile.mkdtemp()\n"
                "    if content: open(os.path.join(d, '_paged_call.so'), 'wb').write(content)\n"
                "    _abi.LIB_PATH = os.path.join(d, 'libkvs.so')\n"
                "    with warnings.catch_warnings(record=True) as w:\n"
                "        warnings.simplefilter('always')\n"
                "        print(paged._load_call(), len(w))\n")
    assert out.splitlines() == ["None 1", "None 1"]
