// MXFP4 x MXFP4 weight products for sm_100a, plain and grouped by expert:
//   Y[m][n] = bf16(sum over 32-column blocks b of 2^(ex[m][b] + ew[n][b]) sum_{k in b} x[m][k] w[n][k])
// with fp32 accumulation in tensor memory (tcgen05.mma kind::mxf4, whose scales
// are read from tensor memory beside the accumulator).
//
// Weight rows are the MMA M dimension (128 a tile), activation rows the MMA N
// dimension (a multiple of 16, at most 240 a tile), so a decoding batch wastes
// no tensor rows and a weight is read once for all the rows of a tile. With
// offsets, expert e's weights meet rows offsets[e] .. offsets[e + 1] only; every
// CTA makes the list of tiles from the offsets itself (they are known on the
// device only) and takes every gridDim-th tile.
//
// Roles (320 threads, a pair's CTAs 384):
//   warps 0-3 epilogue: tensor memory -> registers -> bf16 rows of Y;
//   warp 4    one lane copies the scales into tensor memory (tcgen05.cp) and
//             issues four K = 64 MMAs a block;
//   warps 5,6 bulk copies of the packed weight blocks (codes and scales in one
//             17 KB copy), every other block each: the copy engine serves one
//             issuing thread's copies one after another;
//   warp 7    TMA loads of the activation codes, in the smallest of three box
//             heights that covers the tile's rows;
//   warps 8,9 the activation scales: one word (128 columns) a row. Warp 8 brings
//             them in by TMA as they lie in memory, warp 9 puts them into the
//             order tcgen05.cp reads (lane l, word w: row 32 w + l). They have a
//             ring of their own, so that this step is done ahead of the codes.
//
// Few tiles (p.split > 1): the CTAs of a cluster split a tile's K range, exchange
// their fp32 partials through shared memory and finish a share of the tile's rows
// each, adding the partials in rank order: the result does not depend on timing.
//
// Large products (kPair): two CTAs on two SMs share MMAs of 256 weight rows
// (cta_group::2), each with its own 128 weight rows and half of the activation rows,
// which cuts the bytes a flop moves into shared memory by a third. All copies of a
// pair are counted on the even CTA's barriers; the scales come in the tensor core's
// order from a launch in front. Warps 8-11 are a second set of epilogue warps.
//
// Bound: up to some 250 rows by the weights' way from HBM (0.53 bytes an element:
// 64 experts 2560x5120 at 32 rows 37 us, 0.86 of the measured copy rate; 128 experts
// 2560x2048 at 509 rows 61 us, 0.90), for few weights by the 3.2 us around the blocks
// and a CTA's 0.25 us a block (10240x5120 at one row 8.8 us: 80 CTAs of 20 blocks, since
// the device holds 74 clusters of two and not 80), beyond by the tensor pipe and the
// power cap (51200x5120 at 8192 rows 850 us, 5.0 PFLOP/s; 5120x5120 at 4096 rows 44 us,
// 4.9, and 53 under load), for K of a few blocks by the drain of a pair tile's one
// accumulator beside its products (32 experts 5120x2560 at 32768 rows 250 us, 3.4
// PFLOP/s; the tensor pipe is active for 58 % of a launch, 75 % at twice the K) and the
// L2 (20480x2560 at 16384 rows 10.4 TB/s of tiles in and 1.7 of Y out).
//
// Every wait is bounded (1.5 s); on expiry the kernel records a code in the
// workspace's status word and all roles leave their loops.
#include <cstdint>
#include <cuda_bf16.h>

#include "mx4_internal.h"
#include "mx4_ptx.cuh"
#include "pdl.cuh"
#include "spense.h"

namespace spense {
namespace {

constexpr uint64_t kWaitLimitNs = 1500000000ull;
constexpr int kMaxMx4Stages = 12;
constexpr int kMx4Threads = 320;
constexpr int kMx4PairThreads = 384;
constexpr int kXsSlots = kMx4XsSlots;

struct alignas(16) Mx4Barriers {
  uint64_t full[kMaxMx4Stages];
  uint64_t empty[kMaxMx4Stages];
  uint64_t xs_in[kXsSlots];     // a slot's activation scales have landed, in row order
  uint64_t xs_full[kXsSlots];   // ... are in the tensor core's order
  uint64_t xs_empty[kXsSlots];  // ... are in tensor memory
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Mx4Barriers) <= kMx4BarrierBytes, "barrier area too small");

// kCluster: the barrier is signalled from another CTA too (acquire at cluster scope).
template <bool kCluster = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, unsigned int* status, unsigned int code,
                                         volatile int* abort_flag) {
  auto done = [&] { return kCluster ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity); };
  if (done()) return true;
  const uint64_t t0 = ptx::globaltimer();
  uint32_t it = 0;
  while (true) {
    if (done()) return true;
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
template <bool kCluster = false>
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, unsigned int* status, unsigned int code,
                                         volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_bar<kCluster>(bar, parity, status, code, abort_flag));
}

// Rows [lo, hi) of expert e, for the 32 experts from e0 at once (lane l: e0 + l).
// Offsets are cut to [0, T] and to their running maximum (`carry`, over the calls),
// so ranges never overlap and no offset leads outside the buffers.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int E, int T, int e0, int lane, int& carry, int& lo,
                                            int& hi) {
  const int e = e0 + lane;
  lo = 0;
  hi = e < E ? T : 0;
  if (offsets == nullptr) return;
  int most = e < E ? min(max(ld_dep(offsets + e), 0), T) : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, most, o);
    if (lane >= o) most = max(most, v);
  }
  lo = max(most, carry);
  carry = __shfl_sync(0xffffffffu, lo, 31);
  hi = e < E ? max(min(ld_dep(offsets + e + 1), T), lo) : lo;
}

// Inclusive sum over the warp.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The tile list. tile_begin[e] .. tile_begin[e + 1]: expert e's tiles. first[e],
// count[e]: its rows.
struct TileList {
  int* tile_begin;
  int* first;
  int* count;
};

struct Tile {
  int e, n_tile, row0, rows;
  int row_tile;  // number of the row tile among all experts'
};

template <bool kPair>
__device__ __forceinline__ int weight_tiles(const Mx4GemmParams& p) {
  return kPair ? (p.n_tiles + 1) / 2 : p.n_tiles;
}

// The MMA's N for a tile of so many rows: a multiple of 16, for a pair of 32.
template <bool kPair>
__device__ __forceinline__ int mma_rows(int rows) {
  return kPair ? (rows + 31) & ~31 : (rows + 15) & ~15;
}

template <bool kPair>
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
    // Row tiles in groups of p.group: those of one weight tile next to each other, then
    // the next weight tile's, so that a group's codes stay in L2 while the weights pass.
    const int m_tiles = (cnt + p.npad - 1) / p.npad;
    const int per_group = p.group * weight_tiles<kPair>(p);
    const int group = local / per_group;
    const int in_group = local - group * per_group;
    const int size = min(p.group, m_tiles - group * p.group);
    const int nt = in_group / size;
    const int r = (group * p.group + in_group - nt * size) * p.npad;
    return Tile{__shfl_sync(0xffffffffu, e, 0), __shfl_sync(0xffffffffu, nt, 0),
                __shfl_sync(0xffffffffu, list.first[e] + r, 0), __shfl_sync(0xffffffffu, min(p.npad, cnt - r), 0),
                __shfl_sync(0xffffffffu, list.tile_begin[e] / weight_tiles<kPair>(p) + r / p.npad, 0)};
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

// Stores a warp's 32 weight rows x (8 kGroups) activation rows. Lane l holds the
// bf16 pairs of its weight row, n_warp + l, for activation rows c .. c + 8 kGroups -
// 1. They go through three exchange rounds (with lanes 1, 2 and 4
// apart) that leave each lane with eight consecutive weight rows (8 (l / 8) ..) of
// activation row c + l % 8 of every eight: one 16-byte store a group, 64
// contiguous bytes a row, without shared memory. The rounds of all groups are
// interleaved to cover the exchanges' latency. Where rows of Y are not 16-byte
// aligned, or end in these 32, every lane stores its own values instead, 2 bytes
// each, a warp 64 contiguous bytes of a row.
template <int kGroups>
__device__ __forceinline__ void store_pairs(const uint32_t* a, int lane, uint16_t* y, int64_t ldy, int c, int rows,
                                            int n_warp, int N) {
  if (n_warp + 32 > N || (ldy & 7) != 0) {
    const int n = n_warp + lane;
    uint16_t* dst = y + c * ldy + n;
    if (n < N)
#pragma unroll
      for (int i = 0; i < 8 * kGroups; ++i, dst += ldy)
        if (c + i < rows) *dst = static_cast<uint16_t>(i & 1 ? a[i / 2] >> 16 : a[i / 2] & 0xffffu);
    __syncwarp();
    return;
  }
  const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
  uint32_t q[kGroups][4];
#pragma unroll
  for (int g = 0; g < kGroups; ++g)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t v = a[4 * g + j];
      const uint32_t o = __shfl_xor_sync(0xffffffffu, v, 1);
      q[g][j] = b0 ? __byte_perm(o, v, 0x7632) : __byte_perm(v, o, 0x5410);
    }
  uint32_t r[kGroups][4];
#pragma unroll
  for (int g = 0; g < kGroups; ++g)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, b1 ? q[g][2 * i] : q[g][2 * i + 1], 2);
      r[g][2 * i] = b1 ? o : q[g][2 * i];
      r[g][2 * i + 1] = b1 ? q[g][2 * i + 1] : o;
    }
  const int m = c + (lane & 7);
  uint16_t* dst = y + m * ldy + n_warp + (lane >> 3) * 8;
  uint4 v[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const uint32_t o0 = __shfl_xor_sync(0xffffffffu, b2 ? r[g][0] : r[g][2], 4);
    const uint32_t o1 = __shfl_xor_sync(0xffffffffu, b2 ? r[g][1] : r[g][3], 4);
    v[g] = b2 ? make_uint4(o0, o1, r[g][2], r[g][3]) : make_uint4(r[g][0], r[g][1], o0, o1);
  }
#pragma unroll
  for (int g = 0; g < kGroups; ++g, dst += 8 * ldy)
    if (m + 8 * g < rows) ptx::st_global_v4(dst, v[g]);
}

// The same of fp32 sums.
template <int kGroups>
__device__ __forceinline__ void store_rows(const float* a, int lane, uint16_t* y, int64_t ldy, int c, int rows,
                                           int n_warp, int N) {
  uint32_t pairs[4 * kGroups];
#pragma unroll
  for (int i = 0; i < 4 * kGroups; ++i) pairs[i] = bf16x2(a[2 * i], a[2 * i + 1]);
  store_pairs<kGroups>(pairs, lane, y, ldy, c, rows, n_warp, N);
}

// kBlocks: blocks a stage holds.
template <bool kPair, int kBlocks>
__global__ void __launch_bounds__(kPair ? kMx4PairThreads : kMx4Threads, kPair ? 1 : 2)
    spense_mx4_gemm_kernel(const __grid_constant__ Mx4GemmMaps maps, const __grid_constant__ Mx4GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t smem_base = (raw + 1023u) & ~1023u;  // the swizzled tiles are 1024-byte aligned
  const uint32_t xs_base = smem_base + static_cast<uint32_t>(p.stages) * p.stage_bytes;  // the scales' own ring
  uint8_t* const tail = smem_raw + (xs_base - raw) + (kPair ? 0u : kXsSlots / kBlocks * p.xs_bytes);
  Mx4Barriers* const bars = reinterpret_cast<Mx4Barriers*>(tail);
  TileList list;
  list.tile_begin = reinterpret_cast<int*>(tail + kMx4BarrierBytes);
  list.first = list.tile_begin + p.E + 1;
  list.count = list.first + p.E;
  volatile int* const abort_flag = &bars->abort_flag;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // known to be uniform
  const int lane = threadIdx.x & 31;
  const bool split = !kPair && p.split > 1;
  const uint32_t rank = kPair || split ? ptx::cluster_ctarank() : 0u;
  const int per_unit = kPair ? 2 : p.split;
  const int unit = static_cast<int>(blockIdx.x) / per_unit;  // tiles unit, unit + units, ..
  const int units = static_cast<int>(gridDim.x) / per_unit;
  const int kb0 = kPair ? 0 : static_cast<int>(static_cast<long long>(p.kblocks) * rank / p.split);
  const int kb1 = kPair ? p.kblocks : static_cast<int>(static_cast<long long>(p.kblocks) * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      ptx::mbar_init(ptx::smem_addr(&bars->full[s]), 2);  // weights, activation codes
      ptx::mbar_init(ptx::smem_addr(&bars->empty[s]), 1);
    }
    for (int s = 0; s < kXsSlots; ++s) {
      ptx::mbar_init(ptx::smem_addr(&bars->xs_in[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars->xs_full[s]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars->xs_empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(ptx::smem_addr(&bars->acc_full[a]), 1);
      // pair mode: eight warps of each CTA arrive on the even CTA's
      ptx::mbar_init(ptx::smem_addr(&bars->acc_empty[a]), kPair ? 16 : 128);
    }
    bars->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 4) {
    if constexpr (kPair) {
      ptx::tmem_alloc_pair(ptx::smem_addr(&bars->tmem_base), p.tmem_cols);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(ptx::smem_addr(&bars->tmem_base), p.tmem_cols);
      ptx::tmem_relinquish();
    }
  }
  if (p.offsets != nullptr) ptx::griddep_wait();  // the offsets may be the previous grid's
  if (warp == 0) {
    int begin = 0, carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int lo, hi;
      expert_rows(p.offsets, p.E, p.T, e0, lane, carry, lo, hi);
      const int tiles = (hi - lo + p.npad - 1) / p.npad * weight_tiles<kPair>(p);
      const int scan = warp_scan(tiles, lane);
      if (e < p.E) {
        list.first[e] = lo;
        list.count[e] = hi - lo;
        list.tile_begin[e] = begin + scan - tiles;
      }
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
  if (kPair || split) {
    // The other CTAs' barriers and shared memory are only touched once they have started.
    ptx::cluster_arrive_relaxed();
    ptx::cluster_wait();
  }

  // Activation scales of one column group in a stage: up to 61 rows one narrow
  // box and one tcgen05.cp, else a wide box and one or two.
  const uint32_t group_bytes = kPair || p.npad > 61 ? 1024u : 512u;

  constexpr int bps = kBlocks;  // a stage: the blocks' weights, then their codes
  const uint32_t codes_off = static_cast<uint32_t>(bps) * kMx4BlockBytes;
  const uint32_t xs_slots = static_cast<uint32_t>(kXsSlots / bps);

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
    // Read again by later tiles: kept like the activations (5120x27648 at 16384 rows
    // 1028 us as normal lines, 1006 so).
    const uint64_t pol = p.w_keep ? ptx::policy_evict_last() : ptx::policy_evict_first();
    TileWalker<kPair> walk(p, list);
    Ring ring(static_cast<uint32_t>(p.stages));
    int i = 0;  // stages filled
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile = walk.get(t);
      // Pair mode: the pair's two weight tiles, one a CTA (past the last tile the
      // last one again; those results are not stored).
      const int wt = kPair ? min(2 * tile.n_tile + static_cast<int>(rank), p.n_tiles - 1) : tile.n_tile;
      const int wt0 = (tile.e * p.n_tiles + wt) * p.kblocks;  // the weight tile's first block
      const uint8_t* src = p.blocks + static_cast<size_t>(wt0) * kMx4BlockBytes;
      for (int kb = kb0; kb < kb1; kb += bps, ++i, ring.advance()) {
        if ((i & 1) != (warp & 1)) continue;
        // Nothing is consumed while the previous grid runs, however long that takes.
        if (i >= p.stages && i < p.stages + 2) ptx::griddep_wait();
        ok = wait_all(ptx::smem_addr(&bars->empty[ring.s]), ring.ph ^ 1u, p.status, SPENSE_DEVICE_TIMEOUT_PRODUCER,
                      abort_flag);
        if (!ok) break;
        if (ptx::elect_one()) {
          const uint32_t full = ptx::smem_addr(&bars->full[ring.s]), dst = smem_base + ring.s * p.stage_bytes;
          if constexpr (kPair) {
            // Both CTAs' copies are counted on the even CTA's barrier.
            if (rank == 0) ptx::mbar_arrive_expect_tx(full, 2 * kMx4BlockBytes);
            ptx::tma_load_2d_pair(dst, &maps.w, 0, (wt0 + kb) * (kMx4BlockBytes / 128), ptx::mapa(full, 0u), pol);
          } else {
            const uint32_t bytes = static_cast<uint32_t>(min(bps, kb1 - kb)) * kMx4BlockBytes;
            ptx::mbar_arrive_expect_tx(full, bytes);
            ptx::bulk_g2s(dst, src + static_cast<size_t>(kb) * kMx4BlockBytes, bytes, full, pol);
          }
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
    TileWalker<kPair> walk(p, list);
    Ring ring(static_cast<uint32_t>(p.stages));
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile = walk.get(t);
      // Pair mode: each CTA holds half of the MMA's N rows.
      const int rows = kPair ? mma_rows<kPair>(tile.rows) / 2 : tile.rows;
      const int row0 = tile.row0 + (kPair ? static_cast<int>(rank) * rows : 0);
      const int b = rows <= p.box[0] ? 0 : (rows <= p.box[1] ? 1 : 2);
      const CUtensorMap* map = &maps.x[b];
      const uint32_t bytes = static_cast<uint32_t>(p.box[b]) * 128u;
      for (int kb = kb0; kb < kb1; kb += bps, ring.advance()) {
        ok = wait_all(ptx::smem_addr(&bars->empty[ring.s]), ring.ph ^ 1u, p.status, SPENSE_DEVICE_TIMEOUT_PRODUCER,
                      abort_flag);
        if (!ok) break;
        if (ptx::elect_one()) {
          const uint32_t full = ptx::smem_addr(&bars->full[ring.s]);
          const uint32_t dst = smem_base + ring.s * p.stage_bytes + codes_off;
          if constexpr (kPair) {
            // The scales of all the tile's rows, in the tensor core's order, beside this CTA's half of the codes.
            const uint32_t full0 = ptx::mapa(full, 0u);
            if (rank == 0) ptx::mbar_arrive_expect_tx(full, 2 * (bytes + kMx4XsTileBytes));
            ptx::tma_load_2d_pair(dst, map, kb * 128, row0, full0, pol);
            ptx::tma_load_2d_pair(dst + static_cast<uint32_t>(p.npad / 2) * 128u, &maps.xs_tiles, 0,
                                  (tile.row_tile * p.kblocks + kb) * (kMx4XsTileBytes / 128), full0, pol);
          } else {
            const int nb = min(bps, kb1 - kb);
            ptx::mbar_arrive_expect_tx(full, static_cast<uint32_t>(nb) * bytes);
#pragma unroll
            for (int j = 0; j < kBlocks; ++j)
              if (j < nb)
                ptx::tma_load_2d(dst + static_cast<uint32_t>(j * p.npad) * 128u, map, (kb + j) * 128, row0, full, pol);
          }
        }
      }
    }
  } else if (!kPair && warp == 8) {
    // ------------------------------------------------------------ activation scales in
    // The words of one column group and neighbouring rows, as they lie in memory:
    // one-dimensional boxes of 64 or 256 words from the last 16-byte boundary in
    // front of the tile's first row (words past the array read as zeros).
    test_gate_wait();
    __syncwarp();
    bool ok = __all_sync(0xffffffffu, !*abort_flag);
    ptx::griddep_wait();
    const uint64_t pol = ptx::policy_evict_last();
    TileWalker<kPair> walk(p, list);
    Ring ring(xs_slots);
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile = walk.get(t);
      const bool wide = tile.rows > 61;  // up to three words in front of the tile's rows
      const CUtensorMap* map = wide ? &maps.xs_wide : &maps.xs_narrow;
      for (int kb = kb0; kb < kb1; kb += bps, ring.advance()) {
        ok = wait_all(ptx::smem_addr(&bars->xs_empty[ring.s]), ring.ph ^ 1u, p.status, SPENSE_DEVICE_TIMEOUT_PRODUCER,
                      abort_flag);
        if (!ok) break;
        if (ptx::elect_one()) {
          const uint32_t dst = xs_base + ring.s * p.xs_bytes, bar = ptx::smem_addr(&bars->xs_in[ring.s]);
          const int ng = 2 * min(bps, kb1 - kb);
          ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>(ng) * (wide ? 1024u : 256u));
#pragma unroll
          for (int j = 0; j < 2 * kBlocks; ++j) {
            if (j >= ng) break;
            const int g = min(2 * kb + j, p.groups - 1);  // past the last group the last one again, unused
            ptx::tma_load_1d(dst + static_cast<uint32_t>(j) * group_bytes, map, (g * p.T + tile.row0) & ~3, bar, pol);
          }
        }
      }
    }
  } else if (!kPair && warp == 9) {
    // ------------------------------------------------------------ activation scales into tcgen05.cp's order
    // A warp of its own: the fence in front of the tensor core's reads waits for
    // the memory operations the warp has in flight. Lane l takes rows l, 32 + l, ..
    // of both groups and writes them back as one 16-byte word per 128 rows.
    ptx::griddep_wait();
    TileWalker<kPair> walk(p, list);
    Ring ring(xs_slots);
    bool ok = true;
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile = walk.get(t);
      for (int kb = kb0; kb < kb1; kb += bps, ring.advance()) {
        ok = wait_all(ptx::smem_addr(&bars->xs_in[ring.s]), ring.ph, p.status, SPENSE_DEVICE_TIMEOUT_PRODUCER,
                      abort_flag);
        if (!ok) break;
        uint32_t base = xs_base + ring.s * p.xs_bytes;
        for (int k = kb; k < min(kb + bps, kb1); ++k, base += 2u * group_bytes) {
          const uint32_t s0 = static_cast<uint32_t>(2 * k * p.T + tile.row0) & 3u;
          const uint32_t s1 = static_cast<uint32_t>(min(2 * k + 1, p.groups - 1) * p.T + tile.row0) & 3u;
          uint32_t w[2][8];
#pragma unroll
          for (uint32_t q = 0; q < 8; ++q) {
            if (32 * static_cast<int>(q) >= tile.rows) break;
            const uint32_t at = base + (32u * q + static_cast<uint32_t>(lane)) * 4u;
            w[0][q] = ptx::ld_smem_u32(at + 4u * s0);
            w[1][q] = ptx::ld_smem_u32(at + 4u * s1 + group_bytes);
          }
          __syncwarp();
#pragma unroll
          for (uint32_t j = 0; j < 2; ++j) {
            const uint32_t dst = base + j * group_bytes + static_cast<uint32_t>(lane) * 16u;
            ptx::st_smem_u4(dst, w[j][0], w[j][1], w[j][2], w[j][3]);
            if (tile.rows > 128) ptx::st_smem_u4(dst + 512u, w[j][4], w[j][5], w[j][6], w[j][7]);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&bars->xs_full[ring.s]));
      }
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------ MMA issue
    // The whole warp walks the blocks and one elected lane issues: with control
    // flow the compiler knows to be uniform, the operands stay in uniform
    // registers, where these instructions want them.
    ptx::griddep_wait();  // no bounded wait begins before the activations can come
    TileWalker<kPair> walk(p, list);
    Ring ring(static_cast<uint32_t>(p.stages)), xring(xs_slots);
    const uint32_t sf_base = tmem_base + static_cast<uint32_t>(p.nacc * p.npad);
    const uint32_t atoms = (static_cast<uint32_t>(p.npad) + 127u) >> 7;
    const uint32_t sf_cols = 8u + 8u * atoms;  // of a block: weights' two column groups, activations' two
    uint32_t acc = 0, aph = 1;
    bool ok = !(kPair && rank == 1);  // the even CTA issues the pair's MMAs
    for (int t = unit; ok && t < total; t += units) {
      const Tile tile = walk.get(t);
      const uint32_t idesc = ptx::idesc_mxf4(static_cast<uint32_t>(mma_rows<kPair>(tile.rows)), 0, kPair ? 256u : 128u);
      const uint32_t sf2 = ptx::idesc_mxf4(0, 2) ^ ptx::idesc_mxf4(0, 0);
      ok = wait_all<kPair>(ptx::smem_addr(&bars->acc_empty[acc]), aph, p.status, SPENSE_DEVICE_TIMEOUT_MMA, abort_flag);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t d_tmem = tmem_base + acc * static_cast<uint32_t>(p.npad);
      for (int kb = kb0; kb < kb1; kb += bps, ring.advance(), xring.advance()) {
        ok = (kPair || wait_all(ptx::smem_addr(&bars->xs_full[xring.s]), xring.ph, p.status,
                                SPENSE_DEVICE_TIMEOUT_MMA, abort_flag)) &&
             wait_all(ptx::smem_addr(&bars->full[ring.s]), ring.ph, p.status, SPENSE_DEVICE_TIMEOUT_MMA, abort_flag);
        if (!ok) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const int nb = min(bps, kb1 - kb);
          const uint32_t a_s = smem_base + ring.s * p.stage_bytes;
          auto cp = [](uint32_t taddr, uint64_t desc) {
            if constexpr (kPair)
              ptx::tmem_cp_32x128b_x4_pair(taddr, desc);
            else
              ptx::tmem_cp_32x128b_x4(taddr, desc);
          };
          auto commit = [](uint64_t* bar) {
            if constexpr (kPair)
              ptx::mma_commit_pair(ptx::smem_addr(bar), 0x3);
            else
              ptx::mma_commit(ptx::smem_addr(bar));
          };
          // Every stage has scale columns of its own, so that the stage's refill says
          // that the products that read them have completed.
          const uint32_t sf_stage = sf_base + ring.s * static_cast<uint32_t>(bps) * sf_cols;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            if (b >= nb) break;
            const uint64_t wd = ptx::desc_rows16(a_s + static_cast<uint32_t>(b) * kMx4BlockBytes + kMx4CodeBytes);
            const uint64_t xd = ptx::desc_rows16(kPair ? a_s + kMx4BlockBytes + static_cast<uint32_t>(p.npad / 2) * 128u
                                                       : xs_base + xring.s * p.xs_bytes +
                                                             static_cast<uint32_t>(b) * 2u * group_bytes);
            const uint32_t sfa = sf_stage + static_cast<uint32_t>(b) * sf_cols, sfb = sfa + 8u;
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) {
              cp(sfa + 4u * j, wd + 32u * j);
              cp(sfb + 4u * atoms * j, xd + j * (group_bytes >> 4));
              if (atoms > 1) cp(sfb + 4u * atoms * j + 4u, xd + j * (group_bytes >> 4) + 32u);
            }
          }
          if constexpr (!kPair) commit(&bars->xs_empty[xring.s]);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            if (b >= nb) break;
            const uint64_t ad = ptx::desc_sw128(a_s + static_cast<uint32_t>(b) * kMx4BlockBytes);
            const uint64_t bd = ptx::desc_sw128(a_s + codes_off + static_cast<uint32_t>(b * p.npad) * 128u);
            const uint32_t sfa = sf_stage + static_cast<uint32_t>(b) * sf_cols, sfb = sfa + 8u;
            const uint32_t steps = kb + b + 1 == p.kblocks ? static_cast<uint32_t>(p.last_steps) : 4u;
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
              if (k >= steps) break;
              const uint32_t id = idesc ^ ((k & 1u) ? sf2 : 0u), accum = (kb + b > kb0 || k > 0) ? 1u : 0u;
              const uint32_t fa = sfa + 4u * (k >> 1), fb = sfb + 4u * atoms * (k >> 1);
              if constexpr (kPair)
                ptx::mma_mxf4_pair(d_tmem, ad + 2u * k, bd + 2u * k, id, fa, fb, accum);
              else
                ptx::mma_mxf4(d_tmem, ad + 2u * k, bd + 2u * k, id, fa, fb, accum);
            }
          }
          commit(&bars->empty[ring.s]);
          if (kb + bps >= kb1) commit(&bars->acc_full[acc]);
        }
        __syncwarp();
      }
      if (++acc == static_cast<uint32_t>(p.nacc)) {
        acc = 0;
        aph ^= 1u;
      }
    }
  } else if (warp < 4 || (kPair && warp >= 8)) {
    // ------------------------------------------------------------ epilogue
    constexpr int kEpilogueThreads = kPair ? 256 : 128;
    const int quarter = warp & 3;  // the lanes of tensor memory a warp may read
    ptx::griddep_wait();  // Y may be the previous grid's
    TileWalker<kPair> walk(p, list);
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    int u = 0;
    for (int t = unit; t < total; t += units, ++u) {
      const Tile tile = walk.get(t);
      const uint32_t acc = static_cast<uint32_t>(u % p.nacc), aph = static_cast<uint32_t>((u / p.nacc) & 1);
      if (!ptx::named_bar_and(1, kEpilogueThreads,
                              wait_bar(ptx::smem_addr(&bars->acc_full[acc]), aph, p.status,
                                       SPENSE_DEVICE_TIMEOUT_EPILOGUE, abort_flag)))
        break;
      ptx::tc_fence_after();
      const uint32_t taddr = lane_base + acc * static_cast<uint32_t>(p.npad);
      const int n_warp = (kPair ? 2 * tile.n_tile + static_cast<int>(rank) : tile.n_tile) * kMx4Rows + quarter * 32;
      uint16_t* const y = p.y + static_cast<int64_t>(tile.row0) * p.ldy;
      if (split) break;  // finished below, with the other CTAs of the cluster
      if constexpr (kPair) {
        // Each set of warps takes every other 32 rows, rounds them into registers and
        // gives the accumulator back before its first store: 32 experts 5120x2560 at
        // 32768 rows 272 -> 248 us, where one set of warps gains nothing without and
        // loses with it (310 us). The signal carries no memory access, the reads of
        // tensor memory are complete (wait, fence): relaxed, since a release at cluster
        // scope takes 0.6 us with the accumulator idle (51200x5120 at 8192 rows 906 ->
        // 824 us, at the power cap).
        uint32_t pairs[kMx4PairRows / 4], next[32];
        const int first = warp >= 8 ? 32 : 0;
        if (first < tile.rows) ptx::tmem_ld_32x32b_x32(taddr + static_cast<uint32_t>(first), next);
#pragma unroll
        for (int c = 0; c < kMx4PairRows; c += 64) {
          const int c0 = c + first;
          if (c0 >= tile.rows) break;
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pairs[c / 4 + i] = bf16x2(__uint_as_float(next[2 * i]), __uint_as_float(next[2 * i + 1]));
          if (c0 + 64 < tile.rows) ptx::tmem_ld_32x32b_x32(taddr + static_cast<uint32_t>(c0 + 64), next);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote_relaxed(ptx::mapa(ptx::smem_addr(&bars->acc_empty[acc]), 0u));
#pragma unroll
        for (int c = 0; c < kMx4PairRows; c += 64) {
          const int c0 = c + first;
          if (c0 >= tile.rows) break;
          if (tile.rows - c0 <= 8)
            store_pairs<1>(pairs + c / 4, lane, y, p.ldy, c0, tile.rows, n_warp, p.N);
          else
            store_pairs<4>(pairs + c / 4, lane, y, p.ldy, c0, tile.rows, n_warp, p.N);
        }
        continue;
      }
      // The next 32 rows are read while the ones before are stored.
      uint32_t v[32], next[32];
      ptx::tmem_ld_32x32b_x32(taddr, next);
      for (int c0 = 0; c0 < tile.rows; c0 += 32) {
        ptx::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = next[i];
        if (c0 + 32 < tile.rows) ptx::tmem_ld_32x32b_x32(taddr + static_cast<uint32_t>(c0 + 32), next);
        float a[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) a[i] = __uint_as_float(v[i]);
        if (tile.rows - c0 <= 8)
          store_rows<1>(a, lane, y, p.ldy, c0, tile.rows, n_warp, p.N);
        else
          store_rows<4>(a, lane, y, p.ldy, c0, tile.rows, n_warp, p.N);
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_addr(&bars->acc_empty[acc]));
    }
  }
  __syncwarp();
  if (split) {
    // One tile a cluster at most. The CTAs finish a share of its rows each: `chunk`
    // rows from rank * chunk on. Every thread of the cluster meets here twice: when
    // all MMAs of the cluster have completed, so that every ring is idle and takes
    // the others' partials of its CTA's rows ([source][row / 4][128 weight rows][4
    // rows]), and when they are all in.
    ptx::tc_fence_before();
    ptx::cluster_arrive_relaxed();
    ptx::cluster_wait();
    ptx::tc_fence_after();
    const bool work = warp < 4 && unit < total && !*abort_flag;
    TileWalker<kPair> walk(p, list);
    const Tile tile = work ? walk.get(unit) : Tile{0, 0, 0, 0, 0};
    const uint32_t taddr = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
    const int me = static_cast<int>(rank);
    const int chunk = ((tile.rows + p.split - 1) / p.split + 7) & ~7;
    const uint32_t at = smem_base + static_cast<uint32_t>(warp * 32 + lane) * 16u;
    for (int o = 1; work && o < p.split; ++o) {
      const int r = me + o < p.split ? me + o : me + o - p.split;  // the owner; each source starts with another
      const int r0 = r * chunk, r1 = min(tile.rows, r0 + chunk);
      const uint32_t dst =
          ptx::mapa(at + static_cast<uint32_t>((me < r ? me : me - 1) * chunk) * 512u, static_cast<uint32_t>(r));
      for (int c0 = r0; c0 < r1; c0 += 8) {
        uint32_t v[8];
        ptx::tmem_ld_32x32b_x8(taddr + static_cast<uint32_t>(c0), v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 2; ++q)
          ptx::st_cluster_v4(dst + static_cast<uint32_t>((c0 - r0) / 4 + q) * 2048u,
                             make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                         __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])));
      }
    }
    __syncwarp();
    ptx::cluster_arrive();
    ptx::cluster_wait();
    if (work) {
      const int n_warp = tile.n_tile * kMx4Rows + warp * 32;
      uint16_t* const y = p.y + static_cast<int64_t>(tile.row0) * p.ldy;
      const int r0 = me * chunk, r1 = min(tile.rows, r0 + chunk);
      for (int c0 = r0; c0 < r1; c0 += 8) {
        uint32_t v[8];
        ptx::tmem_ld_32x32b_x8(taddr + static_cast<uint32_t>(c0), v);
        ptx::tmem_ld_wait();
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = 0.0f;
        for (int r = 0; r < p.split; ++r) {  // in rank order, this CTA's own sums among them
          float4 f[2];
          if (r == me) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              f[q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                 __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
          } else {
            const uint32_t src = at + static_cast<uint32_t>((r < me ? r : r - 1) * chunk) * 512u;
#pragma unroll
            for (int q = 0; q < 2; ++q) f[q] = ptx::ld_smem_v4(src + static_cast<uint32_t>((c0 - r0) / 4 + q) * 2048u);
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            a[4 * q] += f[q].x;
            a[4 * q + 1] += f[q].y;
            a[4 * q + 2] += f[q].z;
            a[4 * q + 3] += f[q].w;
          }
        }
        store_rows<1>(a, lane, y, p.ldy, c0, tile.rows, n_warp, p.N);
      }
    }
  }
  if (*abort_flag) {
    // Copies issued before the failure land within microseconds: none may be in
    // flight when the CTA leaves.
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 2000000ull) __nanosleep(1000);
  }
  if (kPair && rank == 1 && warp == 0 && lane == 0) {
    // The even CTA's completion signals land in this CTA's stage barriers
    // asynchronously: wait (bounded) for the last one of every stage. After a
    // failure they may never come; the wait runs out.
    const int my_tiles = unit < total ? (total - unit + units - 1) / units : 0;
    const int items = my_tiles * (kb1 - kb0);
    const uint64_t t0 = ptx::globaltimer();
    for (int i = items > p.stages ? items - p.stages : 0; i < items; ++i) {
      const uint32_t bar = ptx::smem_addr(&bars->empty[i % p.stages]);
      while (!ptx::mbar_try_wait(bar, static_cast<uint32_t>((i / p.stages) & 1)) &&
             ptx::globaltimer() - t0 < kWaitLimitNs) {
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    ptx::tc_fence_after();
    if constexpr (kPair)
      ptx::tmem_dealloc_pair(tmem_base, p.tmem_cols);
    else
      ptx::tmem_dealloc(tmem_base, p.tmem_cols);
  }
  if (kPair) {
    // Neither CTA of a pair leaves while the other may still signal into it.
    ptx::cluster_arrive();
    ptx::cluster_wait();
  }
}

// Pair mode's activation scales: for every row tile and block, the image warp 9
// makes of them in the other mode, so that the pair needs no generic write to
// shared memory that the other CTA's tensor instructions have to see (a release
// at cluster scope took 0.8 us a block). One CTA a row tile and four blocks, all
// of its reads in flight at once: with 16 blocks one after another it took 6.7 us in
// front of 1024 rows of K = 5120 and 16 us in front of K = 27648.
constexpr int kTileThreads = 256;
constexpr int kTilePasses = 2;
constexpr int kTileBlocks = 2 * kTilePasses;

__global__ void __launch_bounds__(kTileThreads)
    mx4_scale_tiles_kernel(const uint32_t* xs, const int32_t* offsets, int E, int T, int npad,
                           int groups, int kblocks, uint32_t* __restrict__ out) {
  ptx::griddep_launch_dependents();
  __shared__ int found[2];
  const int spans = (kblocks + kTileBlocks - 1) / kTileBlocks;
  const int rt = static_cast<int>(blockIdx.x) / spans, kb0 = (static_cast<int>(blockIdx.x) - rt * spans) * kTileBlocks;
  if (threadIdx.x < 2) found[threadIdx.x] = 0;
  ptx::griddep_wait();
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int begin = 0, carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      int lo, hi;
      expert_rows(offsets, E, T, e0, lane, carry, lo, hi);
      const int tiles = (hi - lo + npad - 1) / npad;
      const int scan = warp_scan(tiles, lane);
      const int first = begin + scan - tiles;
      if (rt >= first && rt < first + tiles) {
        found[0] = lo + (rt - first) * npad;
        found[1] = min(npad, hi - found[0]);
      }
      begin += __shfl_sync(0xffffffffu, scan, 31);
    }
  }
  __syncthreads();
  const int row0 = found[0], rows = found[1];
  if (rows == 0) return;  // past the last row tile
  // A thread: four rows 32 apart of one column group, 16 bytes of the image.
  const int lane = threadIdx.x & 31, half = threadIdx.x >> 5 & 1;  // of 128 rows each
  const int r0 = half * 128 + lane;
  uint32_t v[kTilePasses][4];
#pragma unroll
  for (int i = 0; i < kTilePasses; ++i) {
    const int g = 2 * kb0 + 4 * i + (threadIdx.x >> 6);
#pragma unroll
    for (int w = 0; w < 4; ++w)
      v[i][w] = r0 + 32 * w < rows && g < groups ? ld_dep(xs + static_cast<size_t>(g) * T + row0 + r0 + 32 * w) : 0u;
  }
  uint4* dst =
      reinterpret_cast<uint4*>(out) + static_cast<size_t>(rt) * kblocks * (kMx4XsTileBytes / 16) + half * 32 + lane;
#pragma unroll
  for (int i = 0; i < kTilePasses; ++i) {
    const int g = 2 * kb0 + 4 * i + (threadIdx.x >> 6);
    if (g < 2 * kblocks) dst[static_cast<size_t>(g) * 64] = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
  }
}

}  // namespace

cudaError_t launch_mx4_scale_tiles(const Mx4GemmParams& p, int row_tiles, uint32_t* out, cudaStream_t stream) {
  const int spans = (p.kblocks + kTileBlocks - 1) / kTileBlocks;
  return launch_pdl(mx4_scale_tiles_kernel, static_cast<unsigned int>(row_tiles * spans), kTileThreads, 0, stream, p.xs,
                    p.offsets, p.E, p.T, p.npad, p.groups, p.kblocks, out);
}

namespace {

cudaError_t allow_smem() {
  static thread_local int configured_for = -1;
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess || configured_for == dev) return st;
  for (auto f : {spense_mx4_gemm_kernel<false, 1>, spense_mx4_gemm_kernel<false, 2>, spense_mx4_gemm_kernel<true, 1>}) {
    st = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (st != cudaSuccess) return st;
  }
  configured_for = dev;
  return st;
}

cudaLaunchConfig_t gemm_config(int grid, int cluster, uint32_t smem_bytes, cudaStream_t stream,
                               cudaLaunchAttribute (&attr)[3]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(grid));
  cfg.blockDim = dim3(kMx4Threads);
  cfg.dynamicSmemBytes = smem_bytes;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned int>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  attr[2].id = cudaLaunchAttributeClusterSchedulingPolicyPreference;
  attr[2].val.clusterSchedulingPolicyPreference = cudaClusterSchedulingPolicyLoadBalancing;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 3 : 1;
  return cfg;
}

}  // namespace

cudaError_t mx4_max_clusters(int cluster, uint32_t smem_bytes, int* out) {
  cudaError_t st = allow_smem();
  if (st != cudaSuccess) return st;
  cudaLaunchAttribute attr[3];
  const cudaLaunchConfig_t cfg = gemm_config(cluster, cluster, smem_bytes, nullptr, attr);
  return cudaOccupancyMaxActiveClusters(out, spense_mx4_gemm_kernel<false, 1>, &cfg);
}

cudaError_t launch_mx4_gemm(const Mx4GemmMaps& maps, const Mx4GemmParams& p, int grid, uint32_t smem_bytes,
                            cudaStream_t stream) {
  const cudaError_t st = allow_smem();
  if (st != cudaSuccess) return st;
  cudaLaunchAttribute attr[3];
  cudaLaunchConfig_t cfg = gemm_config(grid, p.pair ? 2 : p.split, smem_bytes, stream, attr);
  if (p.pair) {
    cfg.blockDim = dim3(kMx4PairThreads);
    return cudaLaunchKernelEx(&cfg, spense_mx4_gemm_kernel<true, 1>, maps, p);
  }
  return p.bps == 2 ? cudaLaunchKernelEx(&cfg, spense_mx4_gemm_kernel<false, 2>, maps, p)
                    : cudaLaunchKernelEx(&cfg, spense_mx4_gemm_kernel<false, 1>, maps, p);
}

}  // namespace spense
