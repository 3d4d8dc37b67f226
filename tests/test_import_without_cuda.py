"""The package imports, and its host-only calls work, where torch was built without CUDA."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import paged_kv_cache_420_b200 as pkv
assert len(pkv.EXPORTED) > 30 and pkv.version() > 0
assert pkv.lru_victims([3, 1, 2], [1, 1, 0], 2).tolist() == [1, 0]
assert pkv.decode_sparse_workspace_bytes(1, 8, 8, 128, 16, 4) > 0
print("imported")
"""


def test_import_without_torchs_cuda_bindings():
    got = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr[-2000:]
    assert got.stdout.strip() == "imported"
