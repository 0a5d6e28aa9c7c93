"""Calls given a stream of their own, with what they need left for them to make:
the buffers a call makes belong to the stream it runs on. Nothing that the current
stream did before with the same memory, or does with it afterwards, may meet them."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from dense_fp8_gemm_b200 import spense

pytestmark = pytest.mark.gpu

BUSY = 100_000_000  # clock cycles the blocked stream is kept busy: some 50 ms


def mx4_operands(seed, R, K):
    g = np.random.default_rng(seed)
    return [torch.from_numpy(a).cuda() for a in ref.quantize(g.standard_normal((R, K)))]


def mx4_case(M, N, K, E=1):
    wq, ws = mx4_operands(1, E * N, K)
    xq, xs = mx4_operands(2, M, K)
    pw = spense.mx4_pack(wq.view(E, N, -1), ws.view(E, N, -1))
    return pw, xq, torch.from_numpy(ref.words(xs.cpu().numpy())).cuda()


def quantise():
    x = torch.randn(300, 1024, device="cuda").to(torch.bfloat16)
    return lambda stream: spense.mx4_quantize(x, stream=stream)


def dequantise():
    q, s = mx4_operands(3, 300, 1024)
    return lambda stream: (spense.mx4_dequantize(q, s, stream=stream),)


def product():
    pw, xq, xs = mx4_case(1024, 5120, 5120)              # a launch in front orders the scales in the workspace
    return lambda stream: (spense.mx4_gemm(pw, xq, xs, stream=stream),)


def products_of_experts():
    pw, xq, xs = mx4_case(60, 384, 512, E=3)
    off = torch.tensor([0, 20, 20, 60], dtype=torch.int32, device="cuda")
    return lambda stream: (spense.mx4_gemm_experts(pw, xq, xs, off, stream=stream),)


def sort():
    ids = torch.randint(64, (5000, 4), device="cuda")
    return lambda stream: spense.expert_sort(ids, 64, stream=stream)


def combine():
    y = torch.randn(512, 2048, device="cuda").to(torch.bfloat16)
    pos = torch.randperm(512, device="cuda").view(128, 4).to(torch.int32)
    w = torch.rand(128, 4, device="cuda")
    return lambda stream: (spense.expert_combine(y, pos, w, stream=stream),)


MX4 = [quantise, dequantise, product, products_of_experts, sort, combine]


def after_the_past(call):
    """What `call` makes may be memory that the current stream is still about to write."""
    want = [t.clone() for t in call(None)]
    nbytes = [t.untyped_storage().nbytes() for t in call(None)]
    torch.full((1,), 0x55, dtype=torch.uint8, device="cuda")   # a kernel's first launch waits for the GPU
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    torch.cuda._sleep(BUSY)
    past = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in nbytes]
    del past
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("make", MX4)
def test_outputs_made_on_another_stream(make):
    after_the_past(make())


def test_product_keeps_its_workspace_on_another_stream():
    """The workspace a product makes is its own until the product has run there."""
    pw, xq, xs = mx4_case(1024, 5120, 5120)
    y = torch.zeros(1024, 5120, dtype=torch.bfloat16, device="cuda")
    want = spense.mx4_gemm(pw, xq, xs)
    n = spense.mx4_workspace_size(pw, 1024)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    spense.mx4_gemm(pw, xq, xs, Y=y, stream=side)
    later = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in later)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))


def test_sort_keeps_its_counters_on_another_stream():
    M, k, E = 5000, 4, 64
    ids = torch.randint(E, (M, k), device="cuda")
    want = spense.expert_sort(ids, E)
    into = [torch.zeros_like(t) for t in want]
    n = int(spense.lib().spense_expert_sort_workspace_size(M, k, E)) + 4 * (2 * M * k + E + 1)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    spense.expert_sort(ids, E, *into, stream=side)
    later = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in later)
    for a, b in zip(into, want):
        assert torch.equal(a, b)


def fp8_weight(N, K):
    g = torch.Generator(device="cuda").manual_seed(N + K)
    W = (torch.randn(N, K, device="cuda", generator=g)).to(torch.float8_e4m3fn).view(torch.uint8)
    return W, torch.rand(N, device="cuda", generator=g) + 0.5


def fp8_case(M, N, K):
    X, s = fp8_weight(M, K)
    return spense.pack(*fp8_weight(N, K), Kd=K // 4), X, s


def fp8_quantise():
    x = torch.randn(300, 1024, device="cuda").to(torch.bfloat16)
    return lambda stream: spense.quantize(x, stream=stream)


def fp8_product():
    pw, X, s = fp8_case(40, 3000, 2048)
    return lambda stream: (spense.gemm(pw, X, s, stream=stream),)


def fp8_products_in_one_launch():
    pws, X, s = [spense.pack(*fp8_weight(N, 2048), Kd=512) for N in (640, 1500)], *fp8_weight(33, 2048)
    return lambda stream: spense.gemm_grouped(pws, X, s, stream=stream)


def fp8_scores():
    I, H = 1024, 512
    gate, up, down = fp8_weight(I, H), fp8_weight(I, H), fp8_weight(H, I)
    h_in, h_mid = torch.rand(H, device="cuda"), torch.rand(I, device="cuda")
    return lambda stream: (spense.score_glu(*down, h_in, h_mid, *gate, *up, stream=stream),)


def fp8_selection():
    score = torch.rand(4096, device="cuda")
    return lambda stream: (spense.select_dense(score, 1000, stream=stream),)


@pytest.mark.parametrize("make", [fp8_quantise, fp8_product, fp8_products_in_one_launch, fp8_scores, fp8_selection])
def test_fp8_outputs_made_on_another_stream(make):
    after_the_past(make())


def test_fp8_product_keeps_its_workspace_on_another_stream():
    """Partials and counters of tiles that several CTAs share, in a workspace the call makes."""
    pw, X, s = fp8_case(40, 51200, 2048)
    y = torch.zeros(40, 51200, dtype=torch.bfloat16, device="cuda")
    want = spense.gemm(pw, X, s)
    n = spense.workspace_size(pw, 40)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    spense.gemm(pw, X, s, Y=y, stream=side)
    later = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    assert not any(bool(t.any()) for t in later)
    assert torch.equal(y.view(torch.int16), want.view(torch.int16))
