// MXFP4 x MXFP4 weight products for sm_100a, plain and grouped by expert:
//   Y[m][n] = bf16(sum over 32-column blocks b of 2^(ex[m][b] + ew[n][b]) sum_{k in b} x[m][k] w[n][k])
// with fp32 accumulation in tensor memory (tcgen05.mma kind::mxf4, whose scales
// are read from tensor memory beside the accumulator).
//
// Weight rows are the MMA M dimension (128 a tile), activation rows the MMA N
// dimension (a multiple of 16, at most 256 a tile), so a decoding batch wastes
// no tensor rows and a weight is read once for all the rows of a tile. With
// offsets, expert e's weights meet rows offsets[e] .. offsets[e + 1] only; every
// CTA makes the list of tiles from the offsets itself (they are known on the
// device only) and takes every gridDim-th tile, rows of one weight tile next to
// each other so that the weights' second read hits L2.
//
// Roles (320 threads):
//   warps 0-3 epilogue: tensor memory -> registers -> bf16 rows of Y;
//   warp 4    one lane copies the scales into tensor memory (tcgen05.cp) and
//             issues four K = 64 MMAs a block;
//   warps 5,6 bulk copies of the packed weight blocks (codes and scales in one
//             17 KB copy), every other block each: the copy engine serves one
//             issuing thread's copies one after another;
//   warp 7    TMA loads of the activation codes, in the smallest of three box
//             heights that covers the tile's rows;
//   warps 8,9 the activation scales: one word (128 columns) a row. Warp 8 brings
//             them in with 4-byte asynchronous copies (coalesced, since the words
//             of neighbouring rows are neighbours in memory), warp 9 puts them
//             into the order tcgen05.cp reads (lane l, word w: row 32 w + l).
//
// Few tiles (p.split > 1): the CTAs of a cluster split a tile's K range; the
// peers store their fp32 partials into rank 0's shared memory and rank 0 adds
// them in rank order, so the result does not depend on timing.
//
// Every wait is bounded (1.5 s); on expiry the kernel records a code in the
// workspace's status word and all roles leave their loops.
#include <cstdint>
#include <cuda_bf16.h>

#include "mx4_internal.h"
#include "mx4_ptx.cuh"
#include "spense.h"

namespace spense {
namespace {

constexpr uint64_t kWaitLimitNs = 1500000000ull;
constexpr int kMaxMx4Stages = 12;
constexpr int kMx4Threads = 320;

struct alignas(16) Mx4Barriers {
  uint64_t full[kMaxMx4Stages];
  uint64_t empty[kMaxMx4Stages];
  uint64_t xs_in[kMaxMx4Stages];  // a stage's activation scales have landed, in row order
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Mx4Barriers) <= kMx4BarrierBytes, "barrier area too small");

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, unsigned int* status, unsigned int code,
                                         volatile int* abort_flag) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  uint32_t it = 0;
  while (true) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((++it & 63u) == 0) {
      if (*abort_flag) return false;
      if (ptx::globaltimer() - t0 > kWaitLimitNs) {
        atomicOr(status, code);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// The same by a whole (converged) warp, which takes one decision.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, unsigned int* status, unsigned int code,
                                         volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, status, code, abort_flag));
}

// The tile list. tile_begin[e] .. tile_begin[e + 1]: expert e's tiles, its row
// tiles of npad activation rows consecutive for each weight tile. first[e],
// count[e]: its rows. Offsets are cut to [0, T] and to ascending order, so no
// value of theirs leads outside the buffers.
struct TileList {
  int* tile_begin;
  int* first;
  int* count;
};

struct Tile {
  int e, n_tile, row0, rows;
};

struct TileWalker {
  const Mx4GemmParams& p;
  const TileList& list;
  int e;
  __device__ TileWalker(const Mx4GemmParams& pp, const TileList& l) : p(pp), list(l), e(0) {}
  // Tiles are asked for in ascending order, by whole warps (the values pass
  // through a shuffle so that the compiler knows them to be uniform).
  __device__ Tile get(int t) {
    while (t >= list.tile_begin[e + 1]) ++e;
    const int local = t - list.tile_begin[e];
    const int cnt = list.count[e];
    const int m_tiles = (cnt + p.npad - 1) / p.npad;
    const int nt = local / m_tiles;
    const int r = (local - nt * m_tiles) * p.npad;
    return Tile{__shfl_sync(0xffffffffu, e, 0), __shfl_sync(0xffffffffu, nt, 0),
                __shfl_sync(0xffffffffu, list.first[e] + r, 0), __shfl_sync(0xffffffffu, min(p.npad, cnt - r), 0)};
  }
};

struct Ring {
  uint32_t s = 0, ph = 0, n;
  __device__ explicit Ring(uint32_t stages) : n(stages) {}
  __device__ void advance() {
    if (++s == n) {
      s = 0;
      ph ^= 1u;
    }
  }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Stores a warp's 32 weight rows x 8 activation rows. Lane l holds rows c ..
// c + 7 of its weight row as four bf16 pairs; three exchange rounds (with lanes
// 1, 2 and 4 apart) leave it with eight consecutive weight rows (8 (l / 8) ..) of
// activation row c + l % 8: one 16-byte store, 64 contiguous bytes a row. No
// shared memory, and a quarter of the instructions of one store a value.
__device__ __forceinline__ void store_8rows(const uint32_t (&p)[4], int lane, uint16_t* y, int64_t ldy, int c, int rows,
                                            int n_warp, int N) {
  const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t o = __shfl_xor_sync(0xffffffffu, p[j], 1);
    q[j] = b0 ? __byte_perm(o, p[j], 0x7632) : __byte_perm(p[j], o, 0x5410);
  }
  uint32_t r[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t o = __shfl_xor_sync(0xffffffffu, b1 ? q[2 * i] : q[2 * i + 1], 2);
    r[i][0] = b1 ? o : q[2 * i];
    r[i][1] = b1 ? q[2 * i + 1] : o;
  }
  const uint32_t o0 = __shfl_xor_sync(0xffffffffu, b2 ? r[0][0] : r[1][0], 4);
  const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b2 ? r[0][1] : r[1][1], 4);
  const uint4 v = b2 ? make_uint4(o0, o1, r[1][0], r[1][1]) : make_uint4(r[0][0], r[0][1], o0, o1);
  const int m = c + (lane & 7);
  const int n = n_warp + (lane >> 3) * 8;
  if (m >= rows || n >= N) return;
  uint16_t* dst = y + m * ldy + n;
  if (n + 8 <= N && (ldy & 7) == 0) {
    ptx::st_global_v4(dst, v);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < N) dst[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
  }
}

__global__ void __launch_bounds__(kMx4Threads, 2)
    spense_mx4_gemm_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                           const __grid_constant__ CUtensorMap map2, const __grid_constant__ Mx4GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t smem_base = (raw + 1023u) & ~1023u;  // the swizzled tiles are 1024-byte aligned
  uint8_t* const tail = smem_raw + (smem_base - raw) + static_cast<uint32_t>(p.stages) * p.stage_bytes;
  Mx4Barriers* const bars = reinterpret_cast<Mx4Barriers*>(tail);
  TileList list;
  list.tile_begin = reinterpret_cast<int*>(tail + kMx4BarrierBytes);
  list.first = list.tile_begin + p.E + 1;
  list.count = list.first + p.E;
  volatile int* const abort_flag = &bars->abort_flag;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // known to be uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = p.split > 1 ? ptx::cluster_ctarank() : 0u;
  const int unit = static_cast<int>(blockIdx.x) / p.split;  // tiles unit, unit + units, ..
  const int units = static_cast<int>(gridDim.x) / p.split;
  const int kb0 = static_cast<int>(static_cast<long long>(p.kblocks) * rank / p.split);
  const int kb1 = static_cast<int>(static_cast<long long>(p.kblocks) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&bars->full[s]), 3);  // weights, activation codes, activation scales
      ptx::mbar_init(ptx::smem_addr(&bars->empty[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars->xs_in[s]), 32);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(ptx::smem_addr(&bars->acc_full[a]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars->acc_empty[a]), 128);
    }
    bars->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 4) {
    ptx::tmem_alloc(ptx::smem_addr(&bars->tmem_base), p.tmem_cols);
    ptx::tmem_relinquish();
  }
  if (p.offsets != nullptr) ptx::griddep_wait();  // the offsets may be the previous grid's
  if (warp == 0) {
    int begin = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, hi = 0;
      if (e < p.E) {
        lo = 0;
        hi = p.T;
        if (p.offsets != nullptr) {
          lo = min(max(__ldg(p.offsets + e), 0), p.T);
          hi = min(max(__ldg(p.offsets + e + 1), lo), p.T);
        }
        list.first[e] = lo;
        list.count[e] = hi - lo;
      }
      const int tiles = (hi - lo + p.npad - 1) / p.npad * p.n_tiles;
      int scan = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
      }
      if (e < p.E) list.tile_begin[e] = begin + scan - tiles;
      begin += __shfl_sync(0xffffffffu, scan, 31);
    }
    if (lane == 0) list.tile_begin[p.E] = begin;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  // After the tensor memory is taken: a CTA of the next grid on this SM can then
  // not take it first and wait for this grid with it in hand.
  ptx::griddep_launch_dependents();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
  const int total = __shfl_sync(0xffffffffu, list.tile_begin[p.E], 0);
  if (p.split > 1) {
    // Rank 0's shared memory is only written once it has started.
    ptx::cluster_arrive_relaxed();
    ptx::cluster_wait();
  }

  // Activation scales of one column group in a stage: 512 bytes per 128 rows.
  const uint32_t group_bytes = ((static_cast<uint32_t>(p.npad) + 127u) >> 7) * 512u;

  // Test build only (SPENSE_TEST_HOOKS): to exercise the failure path, the
  // loaders wait (bounded) on a word nothing sets, before any copy is issued.
  auto test_gate_wait = [&]() {
#ifdef SPENSE_TEST_HOOKS
    if (lane != 0 || p.test_gate == nullptr) return;
    const uint64_t t0 = ptx::globaltimer();
    while (*reinterpret_cast<const volatile unsigned int*>(p.test_gate) == 0u && !*abort_flag) {
      if (ptx::globaltimer() - t0 > kWaitLimitNs) {
        atomicOr(p.status, SPENSE_DEVICE_TIMEOUT_PRODUCER);
        *abort_flag = 1;
        break;
      }
      __nanosleep(1000);
    }
#endif
  };

  if (warp == 5 || warp == 6) {
    // ------------------------------------------------------------ weights
    test_gate_wait();
    __syncwarp();
    bool ok = __all_sync(0xffffffffu, !*abort_flag);
    const uint64_t pol = p.w_keep ? ptx::policy_evict_normal() : ptx::policy_evict_first();
    TileWalker walk(p, list);
    Ring ring(static_cast<uint32_t>(p.stages));
    int i = 0;
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile = walk.get(t);
      const uint8_t* src =
          p.blocks + (static_cast<size_t>(tile.e) * p.n_tiles + tile.n_tile) * p.kblocks * kMx4BlockBytes;
      for (int kb = kb0; kb < kb1; ++kb, ++i, ring.advance()) {
        if ((i & 1) != (warp & 1)) continue;
        ok = wait_all(ptx::smem_addr(&bars->empty[ring.s]), ring.ph ^ 1u, p.status, SPENSE_DEVICE_TIMEOUT_PRODUCER,
                      abort_flag);
        if (!ok) break;
        if (ptx::elect_one()) {
          const uint32_t full = ptx::smem_addr(&bars->full[ring.s]);
          ptx::mbar_arrive_expect_tx(full, kMx4BlockBytes);
          ptx::bulk_g2s(smem_base + ring.s * p.stage_bytes, src + static_cast<size_t>(kb) * kMx4BlockBytes,
                        kMx4BlockBytes, full, pol);
        }
      }
    }
  } else if (warp == 7) {
    // ------------------------------------------------------------ activation codes
    test_gate_wait();
    __syncwarp();
    bool ok = __all_sync(0xffffffffu, !*abort_flag);
    ptx::griddep_wait();
    const uint64_t pol = ptx::policy_evict_last();
    TileWalker walk(p, list);
    Ring ring(static_cast<uint32_t>(p.stages));
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile = walk.get(t);
      const int b = tile.rows <= p.box[0] ? 0 : (tile.rows <= p.box[1] ? 1 : 2);
      const CUtensorMap* map = b == 0 ? &map0 : (b == 1 ? &map1 : &map2);
      const uint32_t bytes = static_cast<uint32_t>(p.box[b]) * 128u;
      for (int kb = kb0; kb < kb1; ++kb, ring.advance()) {
        ok = wait_all(ptx::smem_addr(&bars->empty[ring.s]), ring.ph ^ 1u, p.status, SPENSE_DEVICE_TIMEOUT_PRODUCER,
                      abort_flag);
        if (!ok) break;
        if (ptx::elect_one()) {
          const uint32_t full = ptx::smem_addr(&bars->full[ring.s]);
          ptx::mbar_arrive_expect_tx(full, bytes);
          ptx::tma_load_2d(smem_base + ring.s * p.stage_bytes + kMx4BlockBytes, map, kb * 128, tile.row0, full, pol);
        }
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ activation scales in
    test_gate_wait();
    ptx::griddep_wait();
    TileWalker walk(p, list);
    Ring ring(static_cast<uint32_t>(p.stages));
    bool ok = __all_sync(0xffffffffu, !*abort_flag);
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile = walk.get(t);
      for (int kb = kb0; kb < kb1; ++kb, ring.advance()) {
        ok = wait_all(ptx::smem_addr(&bars->empty[ring.s]), ring.ph ^ 1u, p.status, SPENSE_DEVICE_TIMEOUT_PRODUCER,
                      abort_flag);
        if (!ok) break;
        const uint32_t dst = smem_base + ring.s * p.stage_bytes + p.xs_off + static_cast<uint32_t>(lane) * 4u;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int g = 2 * kb + j;
          if (g >= p.groups) break;
          const uint32_t* src = p.xs + static_cast<size_t>(g) * p.T + tile.row0;
          for (int r = lane; r < tile.rows; r += 32)
            ptx::cp_async4(dst + j * group_bytes + static_cast<uint32_t>(r - lane) * 4u, src + r);
        }
        ptx::cp_async_arrive(ptx::smem_addr(&bars->xs_in[ring.s]));
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ activation scales into tcgen05.cp's order
    // In place, 128 rows (512 bytes) at a time. A warp of its own: the fence in
    // front of the tensor core's reads waits for the memory operations the warp
    // has in flight, so in the loading warp it put one trip to L2 into every block.
    const int my_tiles = unit < total ? (total - unit + units - 1) / units : 0;
    const int items = my_tiles * (kb1 - kb0);
    Ring ring(static_cast<uint32_t>(p.stages));
    for (int i = 0; i < items; ++i, ring.advance()) {
      if (!wait_all(ptx::smem_addr(&bars->xs_in[ring.s]), ring.ph, p.status, SPENSE_DEVICE_TIMEOUT_PRODUCER,
                    abort_flag))
        break;
      const uint32_t base = smem_base + ring.s * p.stage_bytes + p.xs_off;
      for (uint32_t a = 0; a < 2u * group_bytes; a += 512u) {
        uint32_t w[4];
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) w[q] = ptx::ld_smem_u32(base + a + q * 128u + static_cast<uint32_t>(lane) * 4u);
        __syncwarp();
        ptx::st_smem_u4(base + a + static_cast<uint32_t>(lane) * 16u, w[0], w[1], w[2], w[3]);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&bars->full[ring.s]));
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issue
    // The whole warp walks the blocks and one elected lane issues: with control
    // flow the compiler knows to be uniform, the operands stay in uniform
    // registers, where these instructions want them.
    TileWalker walk(p, list);
    Ring ring(static_cast<uint32_t>(p.stages));
    const uint32_t sf_base = tmem_base + static_cast<uint32_t>(p.nacc * p.npad);
    const uint32_t atoms = (static_cast<uint32_t>(p.npad) + 127u) >> 7;
    uint32_t sbuf = 0, acc = 0, aph = 1;
    bool ok = true;
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile = walk.get(t);
      const uint32_t idesc = ptx::idesc_mxf4((static_cast<uint32_t>(tile.rows) + 15u) & ~15u, 0);
      const uint32_t sf2 = ptx::idesc_mxf4(0, 2) ^ ptx::idesc_mxf4(0, 0);
      ok = wait_all(ptx::smem_addr(&bars->acc_empty[acc]), aph, p.status, SPENSE_DEVICE_TIMEOUT_MMA, abort_flag);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t d_tmem = tmem_base + acc * static_cast<uint32_t>(p.npad);
      for (int kb = kb0; kb < kb1; ++kb, ring.advance()) {
        ok = wait_all(ptx::smem_addr(&bars->full[ring.s]), ring.ph, p.status, SPENSE_DEVICE_TIMEOUT_MMA, abort_flag);
        if (!ok) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint32_t a_s = smem_base + ring.s * p.stage_bytes;
          const uint64_t ad = ptx::desc_sw128(a_s), bd = ptx::desc_sw128(a_s + kMx4BlockBytes);
          const uint64_t wd = ptx::desc_rows16(a_s + kMx4CodeBytes), xd = ptx::desc_rows16(a_s + p.xs_off);
          // Scales: 8 columns for the weights' two column groups, then 8 a group for the activations.
          const uint32_t sfa = sf_base + sbuf * 24u, sfb = sfa + 8u;
          const uint32_t steps = kb + 1 == p.kblocks ? static_cast<uint32_t>(p.last_steps) : 4u;
#pragma unroll
          for (uint32_t j = 0; j < 2; ++j) {
            ptx::tmem_cp_32x128b_x4(sfa + 4u * j, wd + 32u * j);
            ptx::tmem_cp_32x128b_x4(sfb + 8u * j, xd + 32u * j * atoms);
            if (atoms > 1) ptx::tmem_cp_32x128b_x4(sfb + 8u * j + 4u, xd + 32u * j * atoms + 32u);
          }
#pragma unroll
          for (uint32_t k = 0; k < 4; ++k)
            if (k < steps)
              ptx::mma_mxf4(d_tmem, ad + 2u * k, bd + 2u * k, idesc ^ ((k & 1u) ? sf2 : 0u), sfa + 4u * (k >> 1),
                            sfb + 8u * (k >> 1), (kb > kb0 || k > 0) ? 1u : 0u);
          ptx::mma_commit(ptx::smem_addr(&bars->empty[ring.s]));
          if (kb + 1 == kb1) ptx::mma_commit(ptx::smem_addr(&bars->acc_full[acc]));
        }
        __syncwarp();
        sbuf ^= 1u;
      }
      if (++acc == static_cast<uint32_t>(p.nacc)) {
        acc = 0;
        aph ^= 1u;
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    ptx::griddep_wait();  // Y may be the previous grid's
    TileWalker walk(p, list);
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
    int u = 0;
    for (int t = unit; t < total; t += units, ++u) {
      const Tile tile = walk.get(t);
      const uint32_t acc = static_cast<uint32_t>(u % p.nacc), aph = static_cast<uint32_t>((u / p.nacc) & 1);
      if (!ptx::named_bar_and(1, 128,
                              wait_bar(ptx::smem_addr(&bars->acc_full[acc]), aph, p.status,
                                       SPENSE_DEVICE_TIMEOUT_EPILOGUE, abort_flag)))
        break;
      ptx::tc_fence_after();
      const uint32_t taddr = lane_base + acc * static_cast<uint32_t>(p.npad);
      const int n_warp = tile.n_tile * kMx4Rows + warp * 32;
      uint16_t* const y = p.y + static_cast<int64_t>(tile.row0) * p.ldy;
      if (p.split > 1) break;  // finished below, with the other CTAs of the cluster
      for (int c0 = 0; c0 < tile.rows; c0 += 16) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(taddr + static_cast<uint32_t>(c0), v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q[j] = bf16x2(__uint_as_float(v[8 * h + 2 * j]), __uint_as_float(v[8 * h + 2 * j + 1]));
          store_8rows(q, lane, y, p.ldy, c0 + 8 * h, tile.rows, n_warp, p.N);
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_addr(&bars->acc_empty[acc]));
    }
  }
  __syncwarp();
  if (p.split > 1) {
    // One tile a cluster at most. Every thread of the cluster meets here: every
    // MMA of the cluster has completed, so rank 0's ring is idle and takes the
    // peers' partials, [rank - 1][row / 4][128 weight rows][4 rows].
    ptx::tc_fence_before();
    ptx::cluster_arrive();
    ptx::cluster_wait();
    ptx::tc_fence_after();
    const bool work = warp < 4 && unit < total && !*abort_flag;
    TileWalker walk(p, list);
    const Tile tile = work ? walk.get(unit) : Tile{0, 0, 0, 0};
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
    if (work && rank != 0) {
      const uint32_t dst = ptx::mapa(smem_base + (rank - 1u) * static_cast<uint32_t>(p.npad) * 512u +
                                         static_cast<uint32_t>(warp * 32 + lane) * 16u, 0u);
      for (int c0 = 0; c0 < tile.rows; c0 += 16) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(taddr + static_cast<uint32_t>(c0), v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          ptx::st_cluster_v4(dst + static_cast<uint32_t>(c0 / 4 + q) * 2048u,
                             make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                         __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])));
      }
    }
    __syncwarp();
    ptx::cluster_arrive();
    ptx::cluster_wait();
    if (work && rank == 0) {
      const int n_warp = tile.n_tile * kMx4Rows + warp * 32;
      uint16_t* const y = p.y + static_cast<int64_t>(tile.row0) * p.ldy;
      const uint32_t src = smem_base + static_cast<uint32_t>(warp * 32 + lane) * 16u;
      for (int c0 = 0; c0 < tile.rows; c0 += 16) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(taddr + static_cast<uint32_t>(c0), v);
        ptx::tmem_ld_wait();
        float a[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i] = __uint_as_float(v[i]);
        for (int r = 1; r < p.split; ++r) {
          const uint32_t s = src + static_cast<uint32_t>(r - 1) * static_cast<uint32_t>(p.npad) * 512u;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 f = ptx::ld_smem_v4(s + static_cast<uint32_t>(c0 / 4 + q) * 2048u);
            a[4 * q] += f.x;
            a[4 * q + 1] += f.y;
            a[4 * q + 2] += f.z;
            a[4 * q + 3] += f.w;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) q[j] = bf16x2(a[8 * h + 2 * j], a[8 * h + 2 * j + 1]);
          store_8rows(q, lane, y, p.ldy, c0 + 8 * h, tile.rows, n_warp, p.N);
        }
      }
    }
  }
  if (*abort_flag) {
    // Copies issued before the failure land within microseconds: none may be in
    // flight when the CTA leaves.
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 2000000ull) __nanosleep(1000);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

}  // namespace

cudaError_t launch_mx4_gemm(const CUtensorMap (&maps)[3], const Mx4GemmParams& p, int grid, uint32_t smem_bytes,
                            cudaStream_t stream) {
  static thread_local int configured_for = -1;
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess) return st;
  if (configured_for != dev) {
    st = cudaFuncSetAttribute(spense_mx4_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (st != cudaSuccess) return st;
    configured_for = dev;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(grid));
  cfg.blockDim = dim3(kMx4Threads);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned int>(p.split);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  attr[2].id = cudaLaunchAttributeClusterSchedulingPolicyPreference;
  attr[2].val.clusterSchedulingPolicyPreference = cudaClusterSchedulingPolicyLoadBalancing;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 3 : 1;
  return cudaLaunchKernelEx(&cfg, spense_mx4_gemm_kernel, maps[0], maps[1], maps[2], p);
}

}  // namespace spense
