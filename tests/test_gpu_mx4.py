"""MXFP4 quantisation and products on the GPU against a plain 64-bit restatement:
codes and scales bit for bit, products within the fp32 accumulation and the one
bf16 rounding (the bound is derived beside the reference)."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from dense_fp8_gemm_b200 import spense

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def values(seed, M, K, dtype=torch.float32, spread=3):
    """Rows over several magnitudes, with a zero block, ties and one outlier."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((M, K)) * 2.0 ** g.integers(-spread, spread + 1, size=(M, 1))
    x[0, :32] = 0.0
    x[M // 2, K - 32:] = np.resize([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, 4.0, 7.0, -7.9, 6.0], 32)
    x[M - 1, K // 2] = 300.0
    return torch.from_numpy(x).to(dtype)


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def check_quantised(X, q, s):
    rq, rs = ref.quantize(f64(X))
    s = s.cpu().numpy()
    got = s if s.ndim == 2 else ref.rows_of_words(s, X.shape[1])
    assert np.array_equal(got, rs)
    live = np.repeat(rs != 255, 16, axis=1)
    assert np.array_equal(q.cpu().numpy()[live], rq[live])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,K", [(1, 32), (1, 5120), (3, 96), (7, 1056), (8, 1024), (33, 2080), (700, 1184)])
def test_quantize(M, K, dtype):
    X = values(M + K, M, K, DTYPES[dtype]).cuda()
    q, s = spense.mx4_quantize(X)
    check_quantised(X, q, s)
    assert s.shape == (-(-K // 128), M, 4)
    if K % 128:                                              # bytes past the last column are 0
        assert int(s[-1, :, (K % 128) // 32:].max()) == 0
    q2, s2 = spense.mx4_quantize(X, scale_rows=True)
    assert torch.equal(q, q2)
    check_quantised(X, q2, s2)


def test_quantize_extremes():
    """Subnormals, the largest finite values, infinities and NaN."""
    x = torch.zeros((6, 64), dtype=torch.float32)
    x[0, :32] = torch.finfo(torch.float32).max
    x[1, :32] = torch.linspace(-1, 1, 32) * 2.0 ** -126
    x[2, :32] = 2.0 ** -149
    x[3, 5] = float("inf")
    x[4, 40] = float("nan")
    x[5] = torch.linspace(-1, 1, 64) * 2.0 ** -120
    X = x.cuda()
    q, s = spense.mx4_quantize(X)
    check_quantised(X, q, s)
    for dtype in (torch.bfloat16, torch.float32):
        y = f64(spense.mx4_dequantize(q, s, dtype=dtype))
        want = ref.values(q.cpu().numpy(), ref.rows_of_words(s.cpu().numpy(), 64))
        assert np.array_equal(y, want, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [7, 4000])
def test_quantize_every_bit_pattern(dtype, rows):
    """All 65536 patterns of a 16-bit type (subnormals, infinities and NaN among
    them), in blocks of neighbouring patterns and in shuffled ones."""
    bits = np.arange(65536, dtype=np.uint16)
    shuffled = np.random.default_rng(1).permutation(bits)
    both = np.concatenate((bits, shuffled)).reshape(-1, 256)
    x = torch.from_numpy(np.resize(both, (max(rows, 512), 256))[:rows if rows < 512 else None].view(np.int16).copy())
    X = x.cuda().view(DTYPES[dtype])
    q, s = spense.mx4_quantize(X)
    check_quantised(X, q, s)


@pytest.mark.parametrize("M,K", [(1, 32), (5, 160), (40, 1056), (300, 4096)])
@pytest.mark.parametrize("scale_rows", [False, True])
def test_dequantize_every_code(M, K, scale_rows):
    g = np.random.default_rng(M)
    q = g.integers(0, 256, (M, K // 2), dtype=np.uint8)
    s = g.integers(0, 253, (M, K // 32), dtype=np.uint8)
    sd = torch.from_numpy(s if scale_rows else ref.words(s)).cuda()
    want = ref.values(q, s)
    for dtype in (torch.bfloat16, torch.float32):
        y = spense.mx4_dequantize(torch.from_numpy(q).cuda(), sd, dtype=dtype)
        assert y.dtype == dtype and np.array_equal(f64(y), want)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_quantize_gathered_rows(dtype):
    """A gather with repeats; entries outside the rows leave what was there."""
    M, K, T = 37, 352, 300
    X = values(5, M, K, DTYPES[dtype]).cuda()
    g = np.random.default_rng(9)
    rows = g.integers(0, M, T).astype(np.int32)
    rows[[3, 40, 299]] = [-1, M, 2 ** 31 - 1]
    q = torch.full((T, K // 2), 0xAB, dtype=torch.uint8, device="cuda")
    s = torch.full((-(-K // 128), T, 4), 0xCD, dtype=torch.uint8, device="cuda")
    spense.mx4_quantize(X, rows=torch.from_numpy(rows).cuda(), Xq=q, x_scale=s)
    live = (rows >= 0) & (rows < M)
    idx = torch.from_numpy(np.where(live, rows, 0)).long().cuda()
    at = torch.from_numpy(np.flatnonzero(live)).cuda()
    check_quantised(X[idx][at], q[at], s[:, at])
    dead = torch.from_numpy(np.flatnonzero(~live)).cuda()
    assert bool((q[dead] == 0xAB).all()) and bool((s[:, dead] == 0xCD).all())


def test_quantize_strided_rows():
    wide = values(2, 50, 512).cuda()
    X = wide[:, 128:384]
    q, s = spense.mx4_quantize(X)
    check_quantised(X, q, s)


def packed(seed, E, N, K):
    """Weights as codes and scales with the padding's neighbours non-zero."""
    g = np.random.default_rng(seed)
    w = 0.02 * g.standard_normal((E * N, K))
    q, s = ref.quantize(w)
    q, s = q.reshape(E, N, -1), s.reshape(E, N, -1)
    return q, s, spense.mx4_pack(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())


def activations(seed, M, K):
    x = np.random.default_rng(seed + 1000).standard_normal((M, K))
    q, s = ref.quantize(x)
    return q, s, torch.from_numpy(q).cuda(), torch.from_numpy(ref.words(s)).cuda()


def within(y, want, tol):
    err = np.abs(f64(y) - want)
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.size} outside, worst {np.nanmax(err / tol):.3g} bounds"


@pytest.mark.parametrize("N,K", [(1, 32), (128, 256), (130, 288), (300, 1056)])
def test_pack_layout(N, K):
    """Every code and scale byte of the packed blocks is where the header says."""
    E = 2
    q, s, pw = packed(4, E, N, K)
    b = pw.blocks().cpu().numpy()
    nt, kb = -(-N // 128), -(-K // 256)
    assert b.shape == (E, nt, kb, 17408) and pw.weight_bytes == b.size
    codes = np.zeros((E, nt * 128, kb * 128), np.uint8)
    codes[:, :N, :K // 2] = q
    scales = np.zeros((E, nt * 128, kb * 8), np.uint8)
    scales[:, :N, :K // 32] = s
    c = b[..., :16384].reshape(E, nt, kb, 128, 8, 16)
    r = np.arange(128)
    for chunk in range(8):
        want = codes.reshape(E, nt, 128, kb, 8, 16)[:, :, :, :, chunk].transpose(0, 1, 3, 2, 4)
        assert np.array_equal(c[:, :, :, r, chunk ^ (r % 8)], want)
    sc = b[..., 16384:].reshape(E, nt, kb, 2, 32, 4, 4)      # group, lane, word, byte
    want = scales.reshape(E, nt, 4, 32, kb, 2, 4).transpose(0, 1, 4, 5, 3, 2, 6)
    assert np.array_equal(sc, want)
    pw.free()


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 128, 64), (2, 129, 96), (15, 31, 128), (16, 256, 160), (17, 200, 256), (33, 130, 288),
    (64, 1000, 512), (65, 136, 1056), (100, 384, 2048), (128, 128, 320), (129, 264, 544), (200, 72, 1024),
    (256, 640, 768), (257, 129, 256), (520, 392, 832), (45, 640, 8192), (3, 300, 27648), (1, 2560, 5120)])
def test_gemm(M, N, K):
    q, s, pw = packed(M + N, 1, N, K)
    xq, xs, xqd, xsd = activations(K, M, K)
    ws = spense.new_workspace(spense.mx4_workspace_size(pw, M))
    y = spense.mx4_gemm(pw, xqd, xsd, workspace=ws)
    want, tol = ref.gemm(ref.values(xq, xs), ref.values(q[0], s[0]))
    within(y, want, tol)
    again = spense.mx4_gemm(pw, xqd, xsd, workspace=ws)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    assert spense.workspace_status(ws) == 0
    pw.free()


@pytest.mark.parametrize("pad", [0, 3, 8])
def test_gemm_into_a_column_slice(pad):
    M, N, K = 40, 250, 512
    q, s, pw = packed(1, 1, N, K)
    xq, xs, xqd, xsd = activations(2, M, K)
    wide = torch.full((M, N + 16 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    y = wide[:, 8:8 + N]
    spense.mx4_gemm(pw, xqd, xsd, Y=y)
    want, tol = ref.gemm(ref.values(xq, xs), ref.values(q[0], s[0]))
    within(y, want, tol)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + N:] == 7).all())
    pw.free()


def test_gemm_wide_scales():
    """Scales over most of the byte's range, with the products inside bf16's."""
    M, N, K = 20, 140, 256
    g = np.random.default_rng(3)
    q, xq = (g.integers(0, 256, (r, K // 2), dtype=np.uint8) for r in (N, M))
    s, xs = (g.integers(127 - 60, 127 + 60, (r, K // 32)).astype(np.uint8) for r in (N, M))
    pw = spense.mx4_pack(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())
    y = spense.mx4_gemm(pw, torch.from_numpy(xq).cuda(), torch.from_numpy(ref.words(xs)).cuda())
    want, tol = ref.gemm(ref.values(xq, xs), ref.values(q, s))
    within(y, want, tol)
    pw.free()


def test_gemm_nan_scale_stays_in_its_row():
    M, N, K = 33, 200, 512
    q, s, pw = packed(6, 1, N, K)
    xq, xs, xqd, xsd = activations(7, M, K)
    xsd = xsd.clone()
    xsd[1, 5, 2] = 255
    y = f64(spense.mx4_gemm(pw, xqd, xsd))
    want, tol = ref.gemm(ref.values(xq, xs), ref.values(q[0], s[0]))
    assert np.isnan(y[5]).all()
    others = np.arange(M) != 5
    assert (np.abs(y - want)[others] <= tol[others]).all()
    pw.free()


def offsets_of(counts):
    return np.concatenate(([0], np.cumsum(counts))).astype(np.int32)


@pytest.mark.parametrize("counts,spare,N,K", [
    ([5], 0, 128, 256), ([0, 3, 0], 2, 200, 288), ([1] * 9, 0, 130, 512), ([0, 0, 0, 40], 5, 256, 256),
    ([300, 0, 1, 17, 0], 3, 264, 320), ([16, 32, 64, 128, 256, 1], 0, 136, 544), ([0] * 70, 4, 128, 128),
    ([i % 7 for i in range(70)], 0, 384, 1024), ([600, 2], 0, 512, 96), ([2] * 3, 1, 129, 8192)])
def test_gemm_experts(counts, spare, N, K):
    E, T = len(counts), sum(counts) + spare
    q, s, pw = packed(len(counts), E, N, K)
    xq, xs, xqd, xsd = activations(N, T, K)
    off = offsets_of(counts)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = spense.new_workspace(spense.mx4_workspace_size(pw, T))
    spense.mx4_gemm_experts(pw, xqd, xsd, torch.from_numpy(off).cuda(), Y=y, workspace=ws)
    assert spense.workspace_status(ws) == 0
    x = ref.values(xq, xs)
    for e in range(E):
        a, b = off[e], off[e + 1]
        want, tol = ref.gemm(x[a:b], ref.values(q[e], s[e]))
        within(y[a:b], want, tol)
    assert bool((y[off[-1]:] == 7).all())                    # rows behind the last expert's: untouched
    pw.free()


def test_gemm_experts_equals_single_products():
    """Each expert's rows are what spense_mx4_gemm gives for its weight alone."""
    E, N, K, counts = 3, 256, 1024, [20, 0, 50]
    q, s, pw = packed(8, E, N, K)
    _, _, xqd, xsd = activations(9, 70, K)
    y = spense.mx4_gemm_experts(pw, xqd, xsd, torch.from_numpy(offsets_of(counts)).cuda())
    for e, (a, b) in enumerate(((0, 20), (20, 20), (20, 70))):
        one = spense.mx4_pack(torch.from_numpy(q[e]).cuda(), torch.from_numpy(s[e]).cuda())
        if b > a:
            alone = spense.mx4_gemm(one, xqd[a:b].contiguous(), xsd[:, a:b].contiguous())
            assert (f64(alone) == f64(y[a:b])).mean() > 0.99  # the same up to the order of the sums
        one.free()
    pw.free()


def test_offsets_outside_the_rows_are_cut():
    E, N, K, T = 4, 128, 256, 24
    q, s, pw = packed(10, E, N, K)
    xq, xs, xqd, xsd = activations(11, T, K)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([-5, 6, 3, 10, 10 ** 9], dtype=torch.int32, device="cuda")
    spense.mx4_gemm_experts(pw, xqd, xsd, off, Y=y)
    x = ref.values(xq, xs)
    want, tol = ref.gemm(x[10:], ref.values(q[3], s[3]))
    within(y[10:], want, tol)
    want, tol = ref.gemm(x[:3], ref.values(q[0], s[0]))
    within(y[:3], want, tol)
    pw.free()


def test_empty_calls():
    q, s, pw = packed(12, 1, 64, 64)
    y = spense.mx4_gemm(pw, torch.empty((0, 32), dtype=torch.uint8, device="cuda"),
                        torch.empty((1, 0, 4), dtype=torch.uint8, device="cuda"))
    assert y.shape == (0, 64)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    xq, xs = spense.mx4_quantize(x)
    assert xq.shape == (0, 32) and spense.mx4_dequantize(xq, xs).shape == (0, 64)
    pw.free()


def test_pack_rejects_nan_scales():
    q = torch.zeros((4, 32), dtype=torch.uint8, device="cuda")
    s = torch.full((4, 2), 127, dtype=torch.uint8, device="cuda")
    s[3, 1] = 255
    with pytest.raises(spense.SpenseError) as e:
        spense.mx4_pack(q, s)
    assert e.value.code == 6


def device_operands(seed, R, K):
    """Codes and scale bytes drawn on the device (full sizes), scales over eight octaves."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(0, 256, (R, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    s = torch.randint(121, 129, (R, K // 32), dtype=torch.uint8, device="cuda", generator=g)
    return q, s


def words_of(s):
    return torch.nn.functional.pad(s, (0, -s.shape[1] % 4)).view(s.shape[0], -1, 4).permute(1, 0, 2).contiguous()


def check_sampled(y, xq, xs, wq, ws, rows, seed):
    """Sampled rows and columns of a large product (tile borders among them)."""
    g = np.random.default_rng(seed)
    N = wq.shape[0]
    ms = np.unique(np.concatenate((rows[:1], rows[-1:], g.choice(rows, 24))))
    ns = np.unique(np.concatenate(([0, 127, 128, 255, 256, N - 1], g.integers(0, N, 24), [N - 129, N - 128])))
    x = ref.values(xq[ms].cpu().numpy(), xs[ms].cpu().numpy())
    w = ref.values(wq[ns].cpu().numpy(), ws[ns].cpu().numpy())
    want, tol = ref.gemm(x, w)
    within(y[torch.from_numpy(ms).cuda()][:, torch.from_numpy(ns).cuda()], want, tol)


@pytest.mark.parametrize("M,N,K", [(2053, 20001, 5152), (193, 160000, 6656), (4096, 19200, 2592)])
def test_gemm_large_enough_for_pairs(M, N, K):
    assert 2.0 * M * N * K >= 4e11                             # where the plan takes CTA pairs
    wq, ws = device_operands(M, N, K)
    xq, xs = device_operands(N, M, K)
    pw = spense.mx4_pack(wq, ws)
    wsp = spense.new_workspace(spense.mx4_workspace_size(pw, M))
    assert wsp.numel() > 256
    y = spense.mx4_gemm(pw, xq, words_of(xs), workspace=wsp)
    again = spense.mx4_gemm(pw, xq, words_of(xs), workspace=wsp)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    assert spense.workspace_status(wsp) == 0
    check_sampled(y, xq, xs, wq, ws, np.arange(M), M)
    pw.free()


@pytest.mark.parametrize("counts,spare", [([700, 0, 1500], 3), ([1, 2100, 31], 0)])
def test_gemm_experts_large_enough_for_pairs(counts, spare):
    E, T, N, K = len(counts), sum(counts) + spare, 20865, 4640
    assert 2.0 * T * N * K >= 4e11 and T // E >= 512
    wq, ws = device_operands(1, E * N, K)
    xq, xs = device_operands(2, T, K)
    pw = spense.mx4_pack(wq.view(E, N, -1), ws.view(E, N, -1))
    off = offsets_of(counts)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    wsp = spense.new_workspace(spense.mx4_workspace_size(pw, T))
    spense.mx4_gemm_experts(pw, xq, words_of(xs), torch.from_numpy(off).cuda(), Y=y, workspace=wsp)
    assert spense.workspace_status(wsp) == 0
    for e in range(E):
        if counts[e]:
            check_sampled(y, xq, xs, wq[e * N:(e + 1) * N], ws[e * N:(e + 1) * N], np.arange(off[e], off[e + 1]), e)
    assert bool((y[off[-1]:] == 7).all())
    pw.free()


def values_on_device(q, s):
    """ref.values in float64 on the device."""
    lut = torch.from_numpy(np.concatenate((ref.LEVELS, -ref.LEVELS))).to(q.device, torch.float64)
    v = lut[torch.stack((q & 15, q >> 4), -1).long()].view(*s.shape, 32)
    return (v * torch.exp2(s.double() - 127.0)[..., None]).view(s.shape[0], -1)


def check_all(y, xq, xs, wq, ws):
    """Every element of y against ref.gemm's value and tolerance, computed in float64 on the device."""
    x = values_on_device(xq, xs)
    terms = -(-x.shape[1] // 64) + 8
    for n in range(0, wq.shape[0], 4096):
        w = values_on_device(wq[n:n + 4096], ws[n:n + 4096])
        want, acc = x @ w.T, x.abs() @ w.abs().T * (terms * 2.0 ** -23)
        bad = (y[:, n:n + 4096].double() - want).abs() > (want.abs() + acc) * 2.0 ** -8 + acc + 2.0 ** -134
        assert not bool(bad.any()), (n, bad.nonzero()[:4])


@pytest.mark.parametrize("M,N,K", [
    (129, 25601, 2720), (161, 25728, 1184), (200, 25600, 2592), (256, 25600, 2592), (257, 25601, 2592),
    (385, 25600, 1056), (513, 19000, 1056), (700, 19000, 1056), (1024, 5120, 5120), (1100, 4000, 5120),
    (16384, 8192, 160), (8193, 9001, 288), (1500, 10112, 1312), (16000, 2001, 544)])
def test_gemm_tiles_of_pairs(M, N, K):
    """Pair tiles of 160 to 256 rows, full and short, one and several a CTA, over one block of K and more."""
    wq, ws = device_operands(M, N, K)
    xq, xs = device_operands(N, M, K)
    pw = spense.mx4_pack(wq, ws)
    wsp = spense.new_workspace(spense.mx4_workspace_size(pw, M))
    y = spense.mx4_gemm(pw, xq, words_of(xs), workspace=wsp)
    again = spense.mx4_gemm(pw, xq, words_of(xs), workspace=wsp)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    assert spense.workspace_status(wsp) == 0
    check_all(y, xq, xs, wq, ws)
    pw.free()


@pytest.mark.parametrize("N,counts,spare", [
    (20480, [599, 1], 0), (20470, [0, 470, 170], 5), (9000, [0, 256, 257, 255, 1000], 1),
    (8320, [135 + 7 * (i % 5) * (-1) ** i for i in range(20)], 2), (8320, [0, 2700] + [0] * 17 + [192], 0)])
def test_gemm_experts_tiles_of_pairs(N, counts, spare):
    E, T, K = len(counts), sum(counts) + spare, 2592
    wq, ws = device_operands(1, E * N, K)
    xq, xs = device_operands(2, T, K)
    pw = spense.mx4_pack(wq.view(E, N, -1), ws.view(E, N, -1))
    off = offsets_of(counts)
    y = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda")
    wsp = spense.new_workspace(spense.mx4_workspace_size(pw, T))
    spense.mx4_gemm_experts(pw, xq, words_of(xs), torch.from_numpy(off).cuda(), Y=y, workspace=wsp)
    assert spense.workspace_status(wsp) == 0
    for e in range(E):
        a, b = off[e], off[e + 1]
        if b > a:
            check_all(y[a:b], xq[a:b], xs[a:b], wq[e * N:(e + 1) * N], ws[e * N:(e + 1) * N])
    assert bool((y[off[-1]:] == 7).all())
    pw.free()


def test_workspace_serves_fewer_rows():
    """One sized for M rows is enough for every smaller M, whose tiles may be more."""
    N, K = 5120, 1056
    wq, ws = device_operands(3, N, K)
    pw = spense.mx4_pack(wq, ws)
    sizes = [spense.mx4_workspace_size(pw, M) for M in range(2049)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    for top in (128, 700, 1025, 2048):
        wsp = spense.new_workspace(sizes[top])
        for M in (1, top // 3, top // 2 + 1, top - 1, top):
            xq, xs = device_operands(M, M, K)
            y = spense.mx4_gemm(pw, xq, words_of(xs), workspace=wsp)
            check_all(y, xq, xs, wq, ws)
    pw.free()


def test_pairs_on_two_streams_and_captured():
    """Two products in pairs and a small one, on two streams at once, and each stream's sequence as a graph."""
    sets = []
    for i, (M, N, K) in enumerate(((1024, 5120, 5120), (300, 25600, 2592), (5, 640, 1056))):
        wq, ws = device_operands(40 + i, N, K)
        xq, xs = device_operands(50 + i, M, K)
        pw = spense.mx4_pack(wq, ws)
        y = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        wsp = spense.new_workspace(spense.mx4_workspace_size(pw, M))
        sets.append((spense.PreparedMx4Gemm(pw, xq, words_of(xs), y, wsp), y, wsp, (xq, xs, wq, ws)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    order = [[0, 2, 0], [1, 1]]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, todo in zip(streams, order):
            for i in todo:
                sets[i][0](st)
    torch.cuda.synchronize()
    for call, y, wsp, operands in sets:
        check_all(y, *operands)
        assert spense.workspace_status(wsp) == 0
        y.zero_()
    graphs = []
    for st, todo in zip(streams, order):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for i in todo:
                sets[i][0]()
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(10):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for call, y, wsp, operands in sets:
        check_all(y, *operands)
        assert spense.workspace_status(wsp) == 0


def test_small_workspace_is_refused():
    q, s, pw = packed(13, 1, 256, 512)
    _, _, xqd, xsd = activations(14, 5, 512)
    y = torch.empty((5, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(spense.SpenseError) as e:
        spense.mx4_gemm(pw, xqd, xsd, Y=y, workspace=spense.new_workspace(128))
    assert e.value.code == 7
    with pytest.raises(ValueError, match="words"):
        spense.mx4_gemm(pw, xqd, torch.zeros((5, 16), dtype=torch.uint8, device="cuda"), Y=y)
    many = spense.mx4_pack(torch.zeros((2, 8, 32), dtype=torch.uint8, device="cuda"),
                           torch.full((2, 8, 2), 127, dtype=torch.uint8, device="cuda"))
    with pytest.raises(spense.SpenseError) as e:
        spense.mx4_gemm(many, torch.zeros((1, 32), dtype=torch.uint8, device="cuda"),
                        torch.zeros((1, 1, 4), dtype=torch.uint8, device="cuda"))
    assert e.value.code == 1
    with pytest.raises(ValueError, match="offsets"):
        spense.mx4_gemm_experts(many, torch.zeros((1, 32), dtype=torch.uint8, device="cuda"),
                                torch.zeros((1, 1, 4), dtype=torch.uint8, device="cuda"),
                                torch.zeros(2, dtype=torch.int32, device="cuda"))
    many.free()
    pw.free()


def test_two_streams_at_once():
    """Products of two weights on two streams, each with its own workspace, many times over."""
    K, sets = 2048, []
    for i, (M, N) in enumerate(((3, 640), (130, 2560))):
        q, s, pw = packed(20 + i, 1, N, K)
        xq, xs, xqd, xsd = activations(30 + i, M, K)
        y = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        ws = spense.new_workspace(spense.mx4_workspace_size(pw, M))
        want, tol = ref.gemm(ref.values(xq, xs), ref.values(q[0], s[0]))
        sets.append((pw, xqd, xsd, y, ws, want, tol, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(50):
        for pw, xqd, xsd, y, ws, _w, _t, stream in sets:
            spense.mx4_gemm(pw, xqd, xsd, Y=y, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for pw, _x, _s, y, ws, want, tol, _st in sets:
        within(y, want, tol)
        assert spense.workspace_status(ws) == 0
        pw.free()


def test_beside_the_fp8_products_in_one_stream():
    """MXFP4 and FP8 products in turn on one stream (each may start while the other ends)."""
    from dense_fp8_gemm_b200 import synth
    M, N, K = 16, 1024, 2048
    W, s_w = synth.quantize_rows(synth.normal(3, 1, (N, K), 0.02))
    X, s_x = synth.quantize_rows(synth.normal(3, 2, (M, K), 1.0))
    p8 = spense.pack(torch.from_numpy(W).cuda(), torch.from_numpy(s_w).cuda(), Kd=K // 4)
    x8, sx8 = torch.from_numpy(X).cuda(), torch.from_numpy(s_x).cuda()
    w8 = spense.new_workspace(spense.workspace_size(p8, M))
    q, s, p4 = packed(40, 1, N, K)
    xq, xs, xqd, xsd = activations(41, M, K)
    w4 = spense.new_workspace(spense.mx4_workspace_size(p4, M))
    first = spense.gemm(p8, x8, sx8, workspace=w8).clone()
    y8, y4 = torch.empty_like(first), torch.empty_like(first)
    for _ in range(30):
        spense.gemm(p8, x8, sx8, Y=y8, workspace=w8)
        spense.mx4_gemm(p4, xqd, xsd, Y=y4, workspace=w4)
    want, tol = ref.gemm(ref.values(xq, xs), ref.values(q[0], s[0]))
    within(y4, want, tol)
    assert torch.equal(y8.view(torch.int16), first.view(torch.int16))
    p8.free()
    p4.free()
