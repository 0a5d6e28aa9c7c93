"""Scales at the ends of their byte's range: where values and products leave the range
of fp32 and bf16, and where they do not yet."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from dense_fp8_gemm_b200 import spense

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale_rows", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dequantize_at_the_top_of_the_range(dtype, scale_rows):
    """Every code with scale bytes 250 to 255: exact below 2^128, infinite from there on, NaN for 255."""
    q = np.tile((np.arange(16) * 17).astype(np.uint8), (6, 1))      # every code, twice
    s = np.arange(250, 256, dtype=np.uint8)[:, None]
    y = spense.mx4_dequantize(torch.from_numpy(q).cuda(),
                              torch.from_numpy(s if scale_rows else ref.words(s)).cuda(), dtype=dtype)
    want = ref.values(q, s)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    assert np.isinf(want[3]).sum() == 8 and np.isinf(want[4]).sum() == 16 and np.isnan(want[5]).all()
    got = y.double().cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    assert np.array_equal(np.signbit(got[:5]), np.signbit(want[:5]))
