"""Host-side checks of the MXFP4 products' planner (spense_mx4_plan_shapes, no GPU):
every plan fits shared memory, tensor memory and the workspace, covers its rows, and
splits only where the partials find room."""
import random

import pytest

from dense_fp8_gemm_b200 import spense

BLOCK = 17408                  # bytes of a packed block
SMEM = 232448                  # shared memory a CTA can have
TMEM = 512                     # tensor-memory columns of an SM


def bound(E, kblocks, M):
    """What spense_mx4_workspace_size reports for a weight of that shape."""
    grouped = E + M // 128 if M >= 128 * E else 0
    dense = -(-M // 256) + 3 if E == 1 and M >= 128 else 0
    return 256 + max(grouped, dense) * kblocks * 2048


def check(E, N, K, M, grouped, sms):
    p = spense.mx4_plan_shapes(E, N, K, M, grouped, sms)
    n_tiles, kblocks, npad = -(-N // 128), -(-K // 256), p["npad"]
    assert (p["n_tiles"], p["k_blocks"]) == (n_tiles, kblocks)
    pair, split, bps = p["pair"], p["split"], p["blocks_per_stage"]
    # rows a tile takes
    assert npad % (32 if pair else 16) == 0 and 16 <= npad <= (256 if pair else 240)
    if grouped:
        assert p["row_tiles"] >= min(E, M) and p["row_tiles"] * npad >= M
    else:
        assert (p["row_tiles"] - 1) * npad < M <= p["row_tiles"] * npad
    # CTAs: whole pairs, a cluster a tile, or persistent ones
    assert 1 <= p["grid"] <= max(sms, 2) and not (pair and split > 1)   # one CTA an SM
    if pair:
        assert p["grid"] % 2 == 0
    elif split > 1:
        assert 2 <= split <= 8 and p["grid"] == p["row_tiles"] * n_tiles * split and kblocks >= 2 * split
    # shared memory: the ring, the scales' ring, barriers and the tile list
    scales = (2048 if pair else 0)
    assert p["stage_bytes"] == bps * (BLOCK + (npad // 2 if pair else npad) * 128 + scales)
    assert bps == 1 or (npad <= 64 and not pair)
    assert 3 <= p["stages"] <= 12
    fixed = 1024 + 512 + 4 * (3 * E + 1) + (0 if pair else 8 * (2048 if npad > 61 else 1024))
    assert fixed + p["stages"] * p["stage_bytes"] <= p["smem_bytes"] <= SMEM
    # tensor memory: accumulators and every stage's scale columns; more than half of it only alone on an SM
    columns = p["nacc"] * npad + p["stages"] * bps * (24 if npad > 128 else 16)
    assert columns <= p["tmem_cols"] <= TMEM and p["tmem_cols"] & (p["tmem_cols"] - 1) == 0
    assert p["nacc"] in (1, 2) and (split == 1 or p["nacc"] == 1)
    assert p["smem_bytes"] > 233472 // 2       # an SM to itself, whatever its tensor memory
    # a split tile's partials of the other CTAs fit the idle ring
    if split > 1:
        share = -(--(-npad // split) // 8) * 8
        assert (split - 1) * share * 512 <= p["stages"] * p["stage_bytes"]
    # the workspace, and the one a caller asks the size of
    assert p["workspace_bytes"] == 256 + (p["row_tiles"] * kblocks * 2048 if pair else 0)
    assert p["workspace_bytes"] <= bound(E, kblocks, M)
    return p


@pytest.mark.parametrize("N,K", [(1, 32), (128, 256), (2048, 2048), (5120, 5120), (10240, 5120), (5120, 27648),
                                 (51200, 5120), (1 << 20, 96), (64, 1 << 20)])
def test_dense_plans(N, K):
    for M in (1, 2, 15, 16, 17, 45, 64, 65, 127, 128, 129, 200, 240, 241, 256, 257, 700, 1024, 2048, 8191, 16384, 65536):
        for sms in (148, 132, 16):
            check(1, N, K, M, False, sms)
            check(1, N, K, M, True, sms)


@pytest.mark.parametrize("E", [2, 8, 60, 128, 1024])
def test_expert_plans(E):
    for N, K in ((128, 64), (2560, 5120), (5120, 2560), (2560, 2048), (1307, 288)):
        for M in (1, 7, 32, 509, 128 * E - 1, 128 * E, 256 * E - 1, 256 * E, 1 << 17):
            check(E, N, K, M, True, 148)


def test_random_plans():
    rng = random.Random(11)
    for _ in range(4000):
        E = int(2 ** rng.uniform(0, 10))
        N, K, M = int(2 ** rng.uniform(0, 17)), 32 * int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(0, 20))
        if E * -(-N // 128) * -(-K // 256) > 10 ** 7 or M * K > 2 ** 36:
            continue
        check(E, N, K, M, E > 1 or rng.random() < 0.3, 148)


def test_plans_the_measured_shapes_take():
    """One of each kind: pairs where the tensor cores bind, K split where tiles are few, one CTA an SM between."""
    assert check(1, 51200, 5120, 8192, False, 148)["pair"] == 1
    assert check(32, 5120, 2560, 32768, True, 148)["pair"] == 1
    one = check(1, 5120, 5120, 1, False, 148)
    assert one["split"] > 1 and one["pair"] == 0
    batch = check(64, 2560, 5120, 32, True, 148)
    assert batch["split"] == 1 and batch["pair"] == 0 and batch["blocks_per_stage"] == 2


def test_refusals():
    for bad in (dict(E=0), dict(E=1025), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0), dict(K=48), dict(M=0), dict(M=-1),
                dict(M=(1 << 20) + 1), dict(E=1024, N=1 << 20, K=1 << 20)):
        with pytest.raises(spense.SpenseError) as e:
            spense.mx4_plan_shapes(**{**dict(E=2, N=128, K=256, M=4, grouped=True), **bad})
        assert e.value.code == 2, bad
    # a product's words of activation scales: at most 2^31 - 1
    assert spense.mx4_plan_shapes(1, 1, 1 << 20, 262143)["npad"] > 0
    for M, K in ((262144, 1 << 20), (1 << 20, 2048 * 128)):
        with pytest.raises(spense.SpenseError, match="words of activation scales") as e:
            spense.mx4_plan_shapes(1, 1, K, M)
        assert e.value.code == 2
    for bad in (dict(sms=0), dict(sms=1025), dict(E=2, grouped=False)):
        with pytest.raises(spense.SpenseError) as e:
            spense.mx4_plan_shapes(**{**dict(E=1, N=128, K=256, M=4, grouped=True), **bad})
        assert e.value.code == 1, bad
    assert spense.lib().spense_mx4_plan_shapes(1, 128, 256, 4, 0, 148, None) == 1
