"""The package imports, and its host-side checks run, in a torch that was built without CUDA (no GPU)."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)  # such a torch has none of these
import sparse_moe_gemv_b200 as smg
norm = smg.Norm(64)
assert norm.gate_shape(3) == (0,)
try:
    smg.redmoe_norm_forward(norm, torch.zeros(2, 64), x=torch.zeros(2, 64))
except ValueError:
    print("refused")
"""


def test_import_without_cuda_names():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr[-2000:]
