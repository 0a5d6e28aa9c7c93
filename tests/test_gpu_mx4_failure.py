"""The MXFP4 products' waits are bounded: in the test build of the library the
loaders wait on a word nothing sets (SPENSE_TEST_STALL=1), the kernel gives up
after its limit, says so in the status word and returns; the context stays usable.
One child process: the knob is read once. Covers single CTAs, clusters that split K,
CTA pairs and the expert form."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import torch
from dense_fp8_gemm_b200 import spense
def operands(E, N, K, M):
    w = spense.mx4_pack(torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda"),
                        torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda"))
    return (w, torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda"),
            torch.zeros(-(-K // 128), M, 4, dtype=torch.uint8, device="cuda"))
for E, N, K, M in ((1, 128 * 160, 256, 8), (1, 640, 4096, 8), (1, 40960, 2560, 1920), (3, 256, 512, 9)):
    w, xq, xs = operands(E, N, K, M)
    ws = spense.new_workspace(spense.mx4_workspace_size(w, M))
    off = None if E == 1 else torch.tensor([0, 4, 4, 9], dtype=torch.int32, device="cuda")
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    spense.PreparedMx4Gemm(w, xq, xs, y, ws, offsets=off)()
    torch.cuda.synchronize()
    print("RESULT", spense.workspace_status(ws), spense.workspace_status(ws),
          float((torch.ones(1024, device="cuda") * 2).sum().item()))
"""


def test_stalled_loaders_time_out_and_report():
    env = dict(os.environ, SPENSE_TEST_STALL="1", SPENSE_TEST_HOOKS="1")
    r = subprocess.run([sys.executable, "-c", CHILD], env=env, cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    lines = [ln.split() for ln in r.stdout.splitlines() if ln.startswith("RESULT")]
    assert len(lines) == 4
    for _, status, again, usable in lines:
        assert int(status) & 0x1 and int(status) & ~0x7 == 0
        assert int(again) == 0 and float(usable) == 2048.0
