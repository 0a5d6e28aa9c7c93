"""Importing the binding needs no CUDA build of torch (it raises at the first call instead)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):      # as a CPU-only build of torch has it
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from dense_fp8_gemm_b200 import spense
print("VERSION", spense.version())
assert spense.plan_shapes([(1024, 2048, 512)], 16)["tiles"] == 8
try:
    spense.mx4_quantize(torch.zeros(4, 64, dtype=torch.bfloat16))
except (RuntimeError, AssertionError, ValueError, AttributeError) as e:
    print("RAISED", type(e).__name__)
"""


def test_import_without_torch_cuda():
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "VERSION" in r.stdout and "RAISED" in r.stdout
