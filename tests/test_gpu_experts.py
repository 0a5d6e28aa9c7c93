"""The stable sort by expert, the weighted sum of the experts' rows, and a whole
mixture-of-experts layer through the library, against plain restatements."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from dense_fp8_gemm_b200 import spense

pytestmark = pytest.mark.gpu


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def choices(seed, M, k, E, drop):
    g = np.random.default_rng(seed)
    ids = np.minimum(g.exponential(E / 5.0, (M, k)).astype(np.int64), E - 1)
    out = g.random((M, k)) < drop
    ids[out] = g.choice([-1, E, E + 7, -100], out.sum())
    return ids


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("M,k,E,drop", [
    (1, 1, 1, 0.0), (1, 8, 64, 0.0), (3, 2, 5, 0.5), (16, 8, 128, 0.0), (33, 7, 1000, 0.1), (512, 8, 1024, 0.0),
    (513, 8, 256, 0.2), (700, 6, 3, 0.9), (2000, 4, 60, 1.0), (5001, 5, 31, 0.1), (40000, 4, 16, 0.05)])
def test_sort(M, k, E, drop, dtype):
    ids = choices(M + E, M, k, E, drop)
    off, rows, pos = spense.expert_sort(torch.from_numpy(ids).to(dtype).cuda(), E)
    ro, rr, rp = ref.sort(ids, E)
    assert np.array_equal(off.cpu().numpy(), ro)
    assert np.array_equal(rows.cpu().numpy(), rr)
    assert np.array_equal(pos.cpu().numpy(), rp)


def test_sort_wide_ids_do_not_wrap():
    ids = torch.tensor([[2 ** 32 + 1, 1, -2 ** 32, 0]], dtype=torch.int64, device="cuda")
    off, rows, pos = spense.expert_sort(ids, 4)
    assert off.tolist() == [0, 1, 2, 2, 2] and pos.tolist() == [[-1, 1, -1, 0]] and rows.tolist() == [0, 0, -1, -1]


def test_sort_of_nothing():
    off, rows, pos = spense.expert_sort(torch.empty((0, 4), dtype=torch.int64, device="cuda"), 7)
    assert off.tolist() == [0] * 8 and rows.numel() == 0 and pos.shape == (0, 4)


@pytest.mark.parametrize("M,k,N,drop", [(1, 1, 1, 0.0), (3, 2, 8, 0.0), (5, 8, 1000, 0.3), (17, 9, 129, 0.2),
                                        (64, 4, 2560, 0.0), (200, 6, 1023, 0.5), (9, 64, 72, 0.9), (4, 3, 264, 1.0),
                                        (7, 3, 513, 0.1), (6, 5, 1307, 0.2), (33, 1, 1026, 0.0), (5, 2, 2047, 0.3)])
def test_combine(M, k, N, drop):
    g = np.random.default_rng(M + N)
    T = M * k
    y = torch.from_numpy(g.standard_normal((T, N))).to(torch.bfloat16)
    pos = g.permutation(T).reshape(M, k).astype(np.int32)
    w = g.random((M, k)).astype(np.float32)
    out = g.random((M, k)) < drop
    pos[out] = g.choice([-1, T, 2 ** 31 - 1, -2 ** 31], out.sum())
    w[out] = np.nan                                          # a weight that must not be looked at
    got = f64(spense.expert_combine(y.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda()))
    want, tol = ref.combine(f64(y), pos.astype(np.int64), w.astype(np.float64))
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("lo,N,wide", [(0, 64, 64), (8, 64, 80), (8, 61, 75)])
def test_combine_strided(lo, N, wide):
    M, k, T = 6, 3, 30
    g = np.random.default_rng(lo + N)
    buf = torch.from_numpy(g.standard_normal((T, wide))).to(torch.bfloat16).cuda()
    out = torch.full((M, wide), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = g.integers(0, T, (M, k)).astype(np.int32)          # the same row more than once
    w = g.standard_normal((M, k)).astype(np.float32)
    spense.expert_combine(buf[:, lo:lo + N], torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda(),
                          out=out[:, lo:lo + N])
    want, tol = ref.combine(f64(buf[:, lo:lo + N]), pos.astype(np.int64), w.astype(np.float64))
    assert (np.abs(f64(out[:, lo:lo + N]) - want) <= tol).all()
    assert bool((out[:, :lo] == 7).all()) and bool((out[:, lo + N:] == 7).all())


class Layer:
    """A gated mixture-of-experts MLP on static buffers, as a serving loop keeps it."""

    def __init__(self, M, k, E, H, I, seed=0):
        self.M, self.k, self.E, self.H, self.I = M, k, E, H, I
        g = torch.Generator().manual_seed(seed)
        self.gu = torch.randn(E, 2 * I, H, generator=g) * 0.05
        self.dn = torch.randn(E, H, I, generator=g) * 0.05
        self.q = {n: spense.mx4_quantize(w.reshape(-1, w.shape[2]).cuda(), scale_rows=True)
                  for n, w in (("gu", self.gu), ("dn", self.dn))}
        self.p = {n: spense.mx4_pack(c.view(E, -1, c.shape[1]), s.view(E, -1, s.shape[1]))
                  for n, (c, s) in self.q.items()}
        T = M * k
        self.x = torch.zeros(M, H, dtype=torch.bfloat16, device="cuda")
        self.ids = torch.zeros(M, k, dtype=torch.int64, device="cuda")
        self.w = torch.zeros(M, k, device="cuda")
        self.xq = torch.zeros(T, H // 2, dtype=torch.uint8, device="cuda")
        self.xs = torch.zeros(-(-H // 128), T, 4, dtype=torch.uint8, device="cuda")
        self.hid = torch.zeros(T, 2 * I, dtype=torch.bfloat16, device="cuda")
        self.y = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        self.ws = spense.new_workspace(spense.mx4_workspace_size(self.p["gu"], T))

    def __call__(self):
        off, rows, pos = spense.expert_sort(self.ids, self.E)
        spense.mx4_quantize(self.x, rows=rows, Xq=self.xq, x_scale=self.xs)
        spense.mx4_gemm_experts(self.p["gu"], self.xq, self.xs, off, Y=self.hid, workspace=self.ws)
        gate, up = self.hid[:, :self.I].float(), self.hid[:, self.I:].float()
        self.act = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
        self.aq, self.as_ = spense.mx4_quantize(self.act)
        spense.mx4_gemm_experts(self.p["dn"], self.aq, self.as_, off, Y=self.y, workspace=self.ws)
        self.out = spense.expert_combine(self.y, pos, self.w)
        return self.out

    def fill(self, seed, drop):
        g = np.random.default_rng(seed)
        self.x.copy_(torch.from_numpy(g.standard_normal((self.M, self.H))))
        ids = np.argsort(g.random((self.M, self.E)), axis=1)[:, :self.k]
        ids[g.random(ids.shape) < drop] = -1
        self.ids.copy_(torch.from_numpy(ids))
        self.w.copy_(torch.softmax(torch.from_numpy(g.standard_normal((self.M, self.k))), 1))

    def check(self):
        """Each step against 64 bits from the step's own inputs."""
        ids, E = self.ids.cpu().numpy(), self.E
        off, rows, pos = ref.sort(ids, E)
        live = off[-1]
        val = {n: ref.values(c.cpu().numpy(), s.cpu().numpy()).reshape(E, -1, c.shape[1] * 2)
               for n, (c, s) in self.q.items()}
        xq, xs = ref.quantize(f64(self.x)[rows[:live]])
        assert np.array_equal(self.xq[:live].cpu().numpy(), xq)
        for n, x, y in (("gu", ref.values(xq, xs), self.hid),
                        ("dn", ref.values(*ref.quantize(f64(self.act)))[:live], self.y)):
            for e in range(E):
                a, b = off[e], off[e + 1]
                want, tol = ref.gemm(x[a:b], val[n][e])
                assert (np.abs(f64(y[a:b]) - want) <= tol).all(), (n, e)
        want, tol = ref.combine(f64(self.y), pos.astype(np.int64), f64(self.w))
        assert (np.abs(f64(self.out) - want) <= tol).all()
        assert spense.workspace_status(self.ws) == 0


@pytest.mark.parametrize("M,k,E,H,I,drop", [(1, 2, 8, 256, 128, 0.0), (7, 3, 12, 288, 160, 0.3),
                                            (150, 4, 16, 512, 384, 0.1), (5, 2, 4, 256, 128, 1.0)])
def test_layer(M, k, E, H, I, drop):
    layer = Layer(M, k, E, H, I)
    layer.fill(M, drop)
    layer()
    layer.check()


def test_layer_captured_and_replayed():
    """The whole layer in one CUDA graph, replayed on other inputs and routings."""
    layer = Layer(9, 3, 6, 256, 128)
    layer.fill(1, 0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed, drop in ((2, 0.0), (3, 0.5), (4, 1.0)):
        layer.fill(seed, drop)
        graph.replay()
        torch.cuda.synchronize()
        layer.check()
