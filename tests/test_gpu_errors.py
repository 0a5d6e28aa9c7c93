"""What a refused or failed call leaves behind on the GPU side: nothing."""
import ctypes

import pytest
import torch

from dense_fp8_gemm_b200 import spense

pytestmark = pytest.mark.gpu


def test_out_of_memory_is_reported_once():
    """A weight whose packed form (272 GB) no device holds: the call says so, and the error does not stay
    behind for the next calls of this thread, or its next launches, to report as theirs."""
    x = torch.zeros(64, dtype=torch.uint8, device="cuda")   # only its address is taken: nothing is read
    wq, ws = spense.mx4_quantize(torch.ones(8, 64, device="cuda"), scale_rows=True)

    def too_large():
        out = ctypes.c_void_p()
        code = spense.lib().spense_mx4_pack(x.data_ptr(), x.data_ptr(), 1, 1 << 20, 1900 * 256, None, ctypes.byref(out))
        assert code == 8 and out.value is None, code
        assert b"memory" in spense.lib().spense_last_error()

    too_large()
    assert int((torch.zeros(8, device="cuda") + 1).sum().item()) == 8
    spense.mx4_pack(wq, ws).free()
    too_large()
    spense.pack(torch.zeros(16, 256, dtype=torch.uint8, device="cuda"), torch.ones(16, device="cuda"), Kd=64).free()
