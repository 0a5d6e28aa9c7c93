"""Host-only checks of the MXFP4 and expert entry points: every bad argument comes
back as a status code before any device work, and the Python binding refuses what
it can see (no GPU is needed: addresses are never followed)."""
import ctypes

import pytest
import torch

import dense_fp8_gemm_b200.build as build_mod
from dense_fp8_gemm_b200 import spense

ARG, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 1, 2, 3, 7, 11


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return spense.lib()


def no_gpu():
    return not torch.cuda.is_available()


def quantize(L, X=0x1000, x_type=0, M=4, K=64, ldx=64, rows=None, T=4, Xq=0x8000, xs=0x9000, flags=0):
    return L.spense_mx4_quantize(X, x_type, M, K, ldx, rows, T, Xq, xs, flags, None)


def test_quantize_refusals(L):
    assert quantize(L, x_type=3) == ARG and quantize(L, x_type=-1) == ARG
    assert quantize(L, flags=2) == ARG
    assert quantize(L, X=None) == ARG and quantize(L, Xq=None) == ARG and quantize(L, xs=None) == ARG
    for K in (0, 16, 33, 48, (1 << 20) + 32):
        assert quantize(L, K=K, ldx=max(K, 64)) == SHAPE, K
    for M, T in ((-1, -1), ((1 << 20) + 1, (1 << 20) + 1), (4, 5)):
        assert quantize(L, M=M, T=T) == SHAPE, (M, T)
    assert quantize(L, ldx=32) == SHAPE and quantize(L, ldx=(1 << 30) + 8) == SHAPE
    assert quantize(L, rows=0x2000, T=-1) == SHAPE
    assert quantize(L, X=0x1008) == ALIGN and quantize(L, Xq=0x8008) == ALIGN and quantize(L, xs=0x9004) == ALIGN
    assert quantize(L, ldx=68) == ALIGN                       # rows of 136 bytes
    assert quantize(L, x_type=2, ldx=66) == ALIGN and quantize(L, rows=0x2002) == ALIGN


def test_dequantize_refusals(L):
    def call(Xq=0x1000, xs=0x2000, M=4, K=64, Y=0x3000, y_type=0, flags=0):
        return L.spense_mx4_dequantize(Xq, xs, M, K, Y, y_type, flags, None)
    assert call(y_type=1) == ARG and call(y_type=7) == ARG and call(flags=4) == ARG
    assert call(Xq=None) == ARG and call(xs=None) == ARG and call(Y=None) == ARG
    assert call(K=40) == SHAPE and call(M=-1) == SHAPE
    assert call(Xq=0x1004) == ALIGN and call(xs=0x2004) == ALIGN and call(Y=0x3008) == ALIGN


def test_pack_refusals(L):
    def call(Wq=0x1000, ws=0x2000, E=2, N=100, K=64):
        out = ctypes.c_void_p(0x1234)
        code = L.spense_mx4_pack(Wq, ws, E, N, K, None, ctypes.byref(out))
        assert out.value is None
        return code
    assert L.spense_mx4_pack(0x1000, 0x2000, 1, 1, 64, None, None) == ARG
    assert call(Wq=None) == ARG and call(ws=None) == ARG
    for E, N, K in ((0, 100, 64), (1025, 100, 64), (2, 0, 64), (2, (1 << 20) + 1, 64), (2, 100, 0), (2, 100, 72),
                    (1024, 1 << 20, 1 << 20)):
        assert call(E=E, N=N, K=K) == SHAPE, (E, N, K)
    assert call(Wq=0x1008) == ALIGN
    assert L.spense_mx4_free(None) == 0 and L.spense_mx4_get_info(None, None) == ARG
    assert L.spense_mx4_workspace_size(None, 4) == 0


def test_gemm_refuses_null_handles(L):
    assert L.spense_mx4_gemm(None, 0x1000, 0x2000, 4, 0x3000, 64, 0x4000, 256, None) == ARG
    assert L.spense_mx4_gemm_experts(None, 0x1000, 0x2000, 4, 0x5000, 0x3000, 64, 0x4000, 256, None) == ARG
    assert L.spense_mx4_gemm_experts(None, 0x1000, 0x2000, 4, None, 0x3000, 64, 0x4000, 256, None) == ARG
    assert L.spense_mx4_gemm_experts(None, 0x1000, 0x2000, 4, 0x5002, 0x3000, 64, 0x4000, 256, None) == ALIGN


def test_sort_refusals(L):
    def call(ids=0x1000, bits=32, M=4, k=2, E=8, off=0x2000, rows=0x3000, pos=0x4000, ws=0x5000, n=1 << 20):
        return L.spense_expert_sort(ids, bits, M, k, E, off, rows, pos, ws, n, None)
    assert call(bits=16) == ARG
    assert call(ids=None) == ARG and call(off=None) == ARG and call(rows=None) == ARG and call(pos=None) == ARG
    for M, k, E in ((-1, 2, 8), (4, 0, 8), (4, 65, 8), (4, 2, 0), (4, 2, 1025), ((1 << 20) + 1, 1, 8), (1 << 20, 17, 8)):
        assert call(M=M, k=k, E=E) == SHAPE, (M, k, E)
        assert L.spense_expert_sort_workspace_size(M, k, E) == 0
    assert call(ids=0x1002) == ALIGN and call(ids=0x1004, bits=64) == ALIGN and call(pos=0x4001) == ALIGN
    assert call(ws=None) == WORKSPACE and call(n=31) == WORKSPACE and call(ws=0x5010) == ALIGN
    assert L.spense_expert_sort_workspace_size(1 << 20, 16, 1024) >= 4 * 1024 * 128


def test_combine_refusals(L):
    def call(Y=0x1000, T=8, N=64, ldy=64, pos=0x2000, w=0x3000, M=4, k=2, out=0x4000, ldo=64):
        return L.spense_expert_combine(Y, T, N, ldy, pos, w, M, k, out, ldo, None)
    assert call(Y=None) == ARG and call(pos=None) == ARG and call(w=None) == ARG and call(out=None) == ARG
    for bad in (dict(T=-1), dict(T=(1 << 24) + 1), dict(N=0), dict(N=(1 << 20) + 1), dict(M=-1), dict(k=0), dict(k=65),
                dict(ldy=63), dict(ldo=63), dict(ldy=(1 << 30) + 1)):
        assert call(**bad) == SHAPE, bad
    assert call(Y=0x1008) == ALIGN and call(out=0x4002) == ALIGN and call(pos=0x2002) == ALIGN and call(w=0x3001) == ALIGN


@pytest.mark.skipif(not no_gpu(), reason="a GPU is present")
def test_valid_arguments_without_a_device_report_unsupported(L):
    assert quantize(L) == UNSUPPORTED
    assert L.spense_mx4_dequantize(0x1000, 0x2000, 4, 64, 0x3000, 0, 0, None) == UNSUPPORTED
    out = ctypes.c_void_p()
    assert L.spense_mx4_pack(0x1000, 0x2000, 1, 100, 64, None, ctypes.byref(out)) == UNSUPPORTED
    assert L.spense_expert_sort(0x1000, 32, 4, 2, 8, 0x2000, 0x3000, 0x4000, 0x5000, 1 << 20, None) == UNSUPPORTED
    assert L.spense_expert_combine(0x1000, 8, 64, 64, 0x2000, 0x3000, 4, 2, 0x4000, 64, None) == UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_shapes(monkeypatch):
    monkeypatch.setattr(spense, "_device_index", lambda: 0)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        spense.mx4_quantize(x.to(torch.int32))
    with pytest.raises(ValueError, match="current device"):
        spense.mx4_quantize(x)
    with pytest.raises(ValueError):
        spense.mx4_quantize(x[0])
    with pytest.raises(ValueError, match="unit column stride"):
        spense.mx4_quantize(x.t())
    q = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="scales of 4 rows"):
        spense._scale_flags(torch.zeros(4, 3, dtype=torch.uint8), 4, 64)
    with pytest.raises(ValueError):
        spense.mx4_dequantize(q, torch.zeros(4, 2, dtype=torch.uint8), dtype=torch.float16)
    with pytest.raises(ValueError):
        spense.mx4_pack(q, torch.zeros(4, 3, dtype=torch.uint8))
    with pytest.raises(ValueError):
        spense.expert_sort(torch.zeros(4, dtype=torch.int64), 4)
    with pytest.raises(ValueError):
        spense.expert_sort(torch.zeros(4, 2, dtype=torch.float32), 4)
    with pytest.raises(ValueError):
        spense.expert_combine(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 3))


def test_scale_layouts_are_told_apart():
    assert spense._scale_flags(torch.zeros(5, 2, dtype=torch.uint8), 5, 64) == spense.MX4_SCALE_ROWS
    assert spense._scale_flags(torch.zeros(1, 5, 4, dtype=torch.uint8), 5, 64) == 0
