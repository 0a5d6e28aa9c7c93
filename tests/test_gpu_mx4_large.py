"""The MXFP4 and expert calls at the ends of their ranges: 2^20 rows or columns, outputs
and weights whose offsets pass 32 bits, 2^24 choices. Sampled against 64 bits."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from dense_fp8_gemm_b200 import spense

pytestmark = pytest.mark.gpu

TOP = 1 << 20


def operands(seed, R, K):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (R, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    return q, torch.randint(121, 129, (R, K // 32), dtype=torch.uint8, device="cuda", generator=g)


def words_of(s):
    return torch.nn.functional.pad(s, (0, -s.shape[1] % 4)).view(s.shape[0], -1, 4).permute(1, 0, 2).contiguous()


def some(n, seed, ends=2, count=30):
    at = np.concatenate((np.arange(min(ends, n)), n - 1 - np.arange(min(ends, n))))
    return np.unique(np.concatenate((at, np.random.default_rng(seed).integers(0, n, count))))


def check(y, xq, xs, wq, ws, seed):
    ms, ns = some(xq.shape[0], seed), some(wq.shape[0], seed + 1, 1, 60)
    want, tol = ref.gemm(ref.values(xq[ms].cpu().numpy(), xs[ms].cpu().numpy()),
                         ref.values(wq[ns].cpu().numpy(), ws[ns].cpu().numpy()))
    got = y[torch.from_numpy(ms).cuda()][:, torch.from_numpy(ns).cuda()].double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("M,N,K", [(TOP, 4104, 64), (TOP - 77, 1, 32), (3, TOP, 96), (1, TOP, 32), (2, 1, TOP)])
def test_gemm(M, N, K):
    wq, ws = operands(1, N, K)
    xq, xs = operands(2, M, K)
    pw = spense.mx4_pack(wq, ws)
    wsp = spense.new_workspace(spense.mx4_workspace_size(pw, M))
    y = spense.mx4_gemm(pw, xq, words_of(xs), workspace=wsp)
    assert spense.workspace_status(wsp) == 0
    check(y, xq, xs, wq, ws, M)
    pw.free()


@pytest.mark.parametrize("E,N,K,T", [(512, 4096, 4096, 700), (1024, 128, 96, TOP), (7, 4104, 64, TOP)])
def test_gemm_experts(E, N, K, T):
    """4.6 GB of packed weights; the most experts; 4.3e9 outputs."""
    wq, ws = operands(3, E * N, K)
    xq, xs = operands(4, T, K)
    pw = spense.mx4_pack(wq.view(E, N, -1), ws.view(E, N, -1))
    live = T - 5
    off = np.concatenate(([0], np.sort(np.random.default_rng(E).integers(0, live, E - 1)), [live])).astype(np.int32)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    wsp = spense.new_workspace(spense.mx4_workspace_size(pw, T))
    spense.mx4_gemm_experts(pw, xq, words_of(xs), torch.from_numpy(off).cuda(), Y=y, workspace=wsp)
    assert spense.workspace_status(wsp) == 0
    for e in some(E, 5, 2, 8):
        a, b = off[e], off[e + 1]
        if b > a:
            check(y[a:b], xq[a:b], xs[a:b], wq[e * N:(e + 1) * N], ws[e * N:(e + 1) * N], int(e))
    assert bool((y[live:] == 7).all())
    pw.free()


@pytest.mark.parametrize("M,K,T", [(TOP, 4128, 0), (5, 4128, TOP), (TOP, 32, 0), (2, TOP, 0)])
def test_quantize_and_dequantize(M, K, T):
    X = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    rows = torch.randint(-1, M + 1, (T,), device="cuda").to(torch.int32) if T else None
    R = T or M
    q = torch.zeros(R, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.zeros(-(-K // 128), R, 4, dtype=torch.uint8, device="cuda")
    spense.mx4_quantize(X, rows=rows, Xq=q, x_scale=s)
    y = spense.mx4_dequantize(q, s)
    at = torch.from_numpy(some(R, M)).cuda()
    src = rows[at].long() if T else at
    live = ((src >= 0) & (src < M)).cpu().numpy()
    rq, rs = ref.quantize(X[src.clamp(0, M - 1)].double().cpu().numpy())
    assert np.array_equal(q[at].cpu().numpy()[live], rq[live])
    assert np.array_equal(y[at].double().cpu().numpy()[live], ref.values(rq, rs)[live])
    assert not bool(q[at][torch.from_numpy(~live).cuda()].any())


@pytest.mark.parametrize("M,k,E", [(TOP, 16, 1024), ((1 << 24) // 64, 64, 777), (TOP, 1, 1)])
def test_sort(M, k, E):
    ids = torch.randint(-2, E + 2, (M, k), device="cuda")
    off, rows, pos = spense.expert_sort(ids, E)
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    in_order, order = torch.sort(key, stable=True)
    assert torch.equal(off, torch.searchsorted(in_order, torch.arange(E + 1, device="cuda")).to(torch.int32))
    assert torch.equal(rows, torch.where(in_order < E, order // k, -1).to(torch.int32))
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device="cuda")
    assert torch.equal(pos.view(-1), torch.where(key < E, slot, -1).to(torch.int32))


@pytest.mark.parametrize("M,k,N,T", [(TOP, 3, 2600, TOP), (TOP, 2, 2603, TOP), (4, 64, TOP, 300), (4, 64, TOP - 3, 300),
                                     (9, 2, 8, 1 << 24)])
def test_combine(M, k, N, T):
    Y = torch.randn(T, N, device="cuda", dtype=torch.bfloat16)
    pos = torch.randint(-1, T + 1, (M, k), device="cuda").to(torch.int32)
    w = torch.rand(M, k, device="cuda")
    out = spense.expert_combine(Y, pos, w)
    at = torch.from_numpy(some(M, N, 1, 20)).cuda()
    y = Y[pos[at].clamp(0, T - 1).long()].double().cpu().numpy().reshape(-1, N)
    p = pos[at].cpu().numpy()
    mine = np.where((p >= 0) & (p < T), np.arange(p.size).reshape(p.shape), -1)
    want, tol = ref.combine(y, mine, w[at].double().cpu().numpy())
    assert (np.abs(out[at].double().cpu().numpy() - want) <= tol).all()
