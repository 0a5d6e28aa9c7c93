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


@pytest.mark.parametrize("M,N,K", [(16, 128, 64), (70, 300, 2048), (1024, 5120, 5120)])
@pytest.mark.parametrize("codes", [(1, 1), (1, 2), (7, 7), (15, 7)])
def test_products_at_the_ends_of_the_range(M, N, K, codes):
    """One nonzero product a row and column, its two scale bytes from 0 to 254. It has at most four significant
    bits, so fp32 and bf16 hold it as it is from 2^-126 to below 2^128; below, each rounds to its own subnormals
    (steps of 2^-149 and 2^-133), above it is infinite."""
    levels = np.concatenate((ref.LEVELS, -ref.LEVELS))
    ends = np.array([0, 1, 2, 30, 59, 60, 61, 64, 90, 120, 126, 127, 128, 150, 188, 189, 190, 191, 192, 222, 252, 253, 254],
                    np.uint8)
    a, b = np.resize(ends, M), np.resize(ends[::-1], N)
    xq, wq = np.zeros((M, K // 2), np.uint8), np.zeros((N, K // 2), np.uint8)
    xs, ws = np.full((M, K // 32), 127, np.uint8), np.full((N, K // 32), 127, np.uint8)
    at = K - 32                                                # in the last block
    xq[:, at // 2], wq[:, at // 2], xs[:, -1], ws[:, -1] = codes[0], codes[1], a, b
    pw = spense.mx4_pack(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())
    y = spense.mx4_gemm(pw, torch.from_numpy(xq).cuda(), torch.from_numpy(ref.words(xs)).cuda()).double().cpu().numpy()
    want = levels[codes[0]] * levels[codes[1]] * np.exp2(a.astype(np.float64) - 127)[:, None] * \
        np.exp2(b.astype(np.float64) - 127)[None, :]
    large, small = np.abs(want) >= 2.0 ** 128, np.abs(want) < 2.0 ** -126
    assert large.any() and small.any()
    assert np.array_equal(y[large], np.copysign(np.inf, want[large]))
    assert np.array_equal(y[~large & ~small], want[~large & ~small])
    assert (np.abs(y - want)[small] <= 2.0 ** -134 + 2.0 ** -150).all()
    pw.free()


@pytest.mark.parametrize("M", [16, 1024])
def test_zero_codes_stay_zero_at_any_scale(M):
    N, K = 5120, 512
    ends = np.array([0, 1, 127, 253, 254], np.uint8)
    xs, ws = np.resize(ends, (M, K // 32)), np.resize(ends, (N, K // 32))
    full = np.full((N, K // 2), 0x77, np.uint8)
    pw = spense.mx4_pack(torch.from_numpy(full).cuda(), torch.from_numpy(ws).cuda())
    y = spense.mx4_gemm(pw, torch.zeros((M, K // 2), dtype=torch.uint8, device="cuda"),
                        torch.from_numpy(ref.words(xs)).cuda())
    assert not bool(y.any())
    pw.free()
