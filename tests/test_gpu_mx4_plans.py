"""Which plan the MXFP4 products' tests run on, and that the kernel runs the one that is
reported: only CTA pairs leave ordered scales behind the workspace's first 256 bytes."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
from dense_fp8_gemm_b200 import spense

pytestmark = pytest.mark.gpu


def plan(E, N, K, M, grouped=None):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return spense.mx4_plan_shapes(E, N, K, M, E > 1 if grouped is None else grouped, sms)


@pytest.mark.parametrize("M,N,K", [
    (2053, 20001, 5152), (193, 160000, 6656), (4096, 19200, 2592),
    (129, 25601, 2720), (161, 25728, 1184), (200, 25600, 2592), (256, 25600, 2592), (257, 25601, 2592),
    (385, 25600, 1056), (513, 19000, 1056), (700, 19000, 1056), (1024, 5120, 5120), (1100, 4000, 5120),
    (16384, 8192, 160), (8193, 9001, 288), (1500, 10112, 1312), (16000, 2001, 544), (300, 25600, 2592),
    (1920, 40960, 2560)])
def test_shapes_of_the_pair_tests_take_pairs(M, N, K):
    assert plan(1, N, K, M)["pair"] == 1


@pytest.mark.parametrize("E,T,N,K", [(3, 2203, 20865, 4640), (3, 2132, 20865, 4640), (2, 600, 20480, 2592),
                                     (3, 645, 20470, 2592), (5, 1769, 9000, 2592), (20, 2892, 8320, 2592)])
def test_shapes_of_the_expert_pair_tests_take_pairs(E, T, N, K):
    assert plan(E, N, K, T)["pair"] == 1


def test_the_small_tests_split_and_take_two_blocks_a_stage():
    shapes = [(1, 1, 32), (1, 128, 64), (2, 129, 96), (15, 31, 128), (16, 256, 160), (17, 200, 256), (33, 130, 288),
              (64, 1000, 512), (65, 136, 1056), (100, 384, 2048), (128, 128, 320), (129, 264, 544), (200, 72, 1024),
              (256, 640, 768), (257, 129, 256), (520, 392, 832), (45, 640, 8192), (3, 300, 27648), (1, 2560, 5120)]
    plans = [plan(1, N, K, M) for M, N, K in shapes]
    assert {p["split"] for p in plans} >= {1, 8} and all(p["blocks_per_stage"] == 2 for p in plans)


@pytest.mark.parametrize("E,T,N,K,npad", [(5, 321, 264, 320, 144), (6, 493, 136, 544, 176), (2, 602, 512, 96, 208)])
def test_the_expert_tests_take_wide_tiles(E, T, N, K, npad):
    p = plan(E, N, K, T)
    assert (p["npad"], p["pair"], p["blocks_per_stage"]) == (npad, 0, 1)


@pytest.mark.parametrize("M,N,K,kind", [
    (1024, 5120, 5120, dict(pair=1)), (2000, 10240, 1056, dict(pair=1)),
    (16, 40960, 512, dict(pair=0, split=1, blocks_per_stage=2, nacc=2)),
    (120, 19000, 1056, dict(pair=0, split=1, blocks_per_stage=1, npad=128)),
    (110, 37000, 1056, dict(pair=0, split=1, blocks_per_stage=1, npad=112)),
    (40, 256, 8192, dict(pair=0, split=8, blocks_per_stage=2)), (130, 2560, 5120, dict(pair=0, split=3, npad=80)),
    (230, 640, 8192, dict(pair=0, split=8, blocks_per_stage=1)), (45, 5120, 5120, dict(pair=0, split=3))])
def test_the_kernel_runs_the_reported_plan(M, N, K, kind):
    p = plan(1, N, K, M)
    assert {k: p[k] for k in kind} == kind, p
    g = np.random.default_rng(M)
    wq, ws = ref.quantize(0.02 * g.standard_normal((N, K)))
    xq, xs = ref.quantize(g.standard_normal((M, K)))
    pw = spense.mx4_pack(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())
    assert spense.mx4_workspace_size(pw, M) >= p["workspace_bytes"]
    wsp = spense.new_workspace(spense.mx4_workspace_size(pw, M))
    y = spense.mx4_gemm(pw, torch.from_numpy(xq).cuda(), torch.from_numpy(ref.words(xs)).cuda(), workspace=wsp)
    assert spense.workspace_status(wsp) == 0
    assert bool(wsp[256:].any()) == bool(p["pair"])
    assert not bool(wsp[p["workspace_bytes"]:].any())
    ms, ns = g.integers(0, M, 40), g.integers(0, N, 200)
    want, tol = ref.gemm(ref.values(xq[ms], xs[ms]), ref.values(wq[ns], ws[ns]))
    got = y[torch.from_numpy(ms).cuda()][:, torch.from_numpy(ns).cuda()].double().cpu().numpy()
    assert (np.abs(got - want) <= tol).all()
    pw.free()


def test_workspace_size_refuses_what_the_products_refuse():
    """More words of activation scales than 32 bits count."""
    K = 1 << 20
    pw = spense.mx4_pack(torch.zeros((1, K // 2), dtype=torch.uint8, device="cuda"),
                         torch.full((1, K // 32), 127, dtype=torch.uint8, device="cuda"))
    assert spense.mx4_workspace_size(pw, 262143) > 256
    for M in (262144, 1 << 20):
        with pytest.raises(spense.SpenseError, match="words of activation scales"):
            spense.mx4_workspace_size(pw, M)
        assert spense.lib().spense_mx4_gemm(pw.handle, 0x1000, 0x1000, M, 0x1000, 1, 0x1000, 1 << 40, None) == 2
    pw.free()
