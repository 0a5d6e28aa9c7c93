"""Kernels that may start while the grid before them still runs read what that grid
writes by coherent loads only (a source check: no result that can be provoked shows
the difference)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp8_gemm_b200", "csrc")


def functions(text):
    """Top-level device functions: from a line that opens one to the brace in the first column that closes it."""
    return re.findall(r"^(?:template[^\n]*\n)?(?:__global__|__device__)[^;{]*\{.*?^\}", text, re.M | re.S)


@pytest.mark.parametrize("name", ["experts.cu", "mx4_gemm.cu", "mx4_quant.cu"])
def test_kernels_that_start_early_use_no_non_coherent_loads(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    bodies = functions(text)
    early = [b for b in bodies if re.search(r"pdl_wait\(|griddep_wait\(", b)]
    assert early
    for body in early + [b for b in bodies if "__global__" not in b]:
        head = body[:body.index("{")]
        assert not re.search(r"const\s+\w+\*\s*__restrict__", head), head
        assert not re.search(r"__ld(g|cg|ca|cs|lu)\(|ld\.global\.nc", body), head
