"""The package on a torch built without GPU support: it imports, and its host-only calls work."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)      # such a build has none of them
import fft_causal_long_amd as sc
assert sc.sc_version() >= 902 and sc.sc_workspace_bytes(sc.KIND_F32, 1, 1, 65536) > 0
x = torch.zeros(4, 8)
try:
    sc.layer_norm(x)
except ValueError:
    print("refused")
"""


def test_import_without_gpu_entry_points():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip().endswith("refused")
