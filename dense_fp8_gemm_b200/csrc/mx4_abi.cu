// C entry points of the MXFP4 and expert operators: argument validation, the
// packed handle and launch planning.
#include <algorithm>
#include <array>
#include <atomic>
#include <climits>
#include <cstdlib>
#include <new>

#include "abi_util.h"
#include "mx4_internal.h"

using namespace spense;

struct spense_mx4_packed {
  int device = -1;
  int64_t E = 0, N = 0, K = 0;
  int n_tiles = 0, kblocks = 0;
  uint8_t* blocks = nullptr;
};

namespace {

constexpr size_t kMx4Header = 256;  // workspace: status word, then pair mode's scale tiles

constexpr uint32_t kMx4Smem = 232448u;  // shared memory of a CTA, which has its SM to itself

// Clusters of s CTAs that the current device holds at once (148 SMs: 74, 45, 33, 26, 22,
// 15 and 15 of 2 to 8); without it (`ask` false) an estimate for so many SMs.
int clusters_at_once(int s, int sms, bool ask) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][9];  // the number + 1; 0: not asked yet
  int dev = -1;
  const int estimate = 10 * sms / (11 * s);
  if (!ask || cudaGetDevice(&dev) != cudaSuccess) return estimate;
  if (dev < kDevices && known[dev][s] > 0) return known[dev][s] - 1;
  int n = 0;
  if (mx4_max_clusters(s, kMx4Smem, &n) != cudaSuccess) {
    cudaGetLastError();
    return estimate;
  }
  if (dev < kDevices) known[dev][s] = n + 1;
  return n;
}

// Estimated time of a launch, in microseconds, from measured rates of this
// kernel: a CTA takes 0.27 us a block and 0.0006 more a row of the tile (latency
// of its ring), all CTAs together 12.4 TB/s from L2 and the weights 5.5 TB/s from
// HBM; 3.2 us go before and after the blocks, 6 ns a row into the epilogue, 0.8 us and
// 12 ns a row into the exchange of a split tile's partials. Against a sweep of 5
// shapes x 7 row counts (M 1 .. 1024) x tiles x splits the choices by it are within
// 20 % of the best.
double mx4_cost(int n, int split, int64_t tiles, int kblocks, double weight_bytes, int sms) {
  const int64_t ctas = tiles * split;
  const double waves = static_cast<double>((tiles + sms - 1) / sms);
  const double blocks = split == 1 ? waves * kblocks : (kblocks + split - 1) / split;
  const double l2 = (kMx4BlockBytes + n * 136.0) * static_cast<double>(std::min<int64_t>(ctas, sms)) / 12.4e6;
  const double block = std::max(0.27 + 0.0006 * n, l2);
  const double t = 3.2 + 0.006 * n + blocks * block + (split > 1 ? 0.8 + 0.012 * n : 0.0);
  return std::max(t, 3.2 + weight_bytes / 5.5e6) + 0.05 * t;
}

// Rows a tile of activations takes, CTA pairs, cluster split, ring depth.
//
// A tile reads its weight block and its activation rows for every 256 columns of
// K. Dense products: rows in equal tiles of at most 240, as many as mx4_cost
// likes. With experts the device alone knows who has how many rows: room for
// twice the average, since a heavier expert only costs a second reading of its
// weights (from L2) and smaller tiles leave a deeper ring.
//
// Few tiles: clusters of up to 8 CTAs split K, when the device holds all of them
// at once and their partials fit the ring.
//
// Pairs: 256 weight rows and up to 256 activation rows by two SMs. They read up to a
// third fewer bytes from L2 for the same products, but a launch in front orders their
// scales and both CTAs fill before the first product. Dense products take whichever
// mx4_cost and mx4_pair_cost call cheaper (singles against pairs: 51200x5120 at 128,
// 256 and 1024 rows 27 -> 28, 52 -> 36 and 149 -> 120 us, 5120x5120 at 1024 and 4096
// rows 19.5 -> 18.6 and 64 -> 51, 8192x1408 at 2048 rows 31 -> 25, 8192x256 at 16384
// rows 117 -> 107). With experts pairs take 256 rows a tile from 256 rows on average
// and 5e10 flops on (128 x 2560x2048 at 256 rows each 166 -> 144 us, 4 x 10240x5120 at
// 256 rows 48 -> 42, 8 x 8192x512 at 1024 rows 68 -> 67), and 192, which leaves tensor
// memory for two accumulators, from 128 rows and 1e11 flops on (128 x 2560x2048 at 128
// rows 101 -> 94 us, at 64 rows 76 -> 78; 8 x 5120x5120 at 128 rows 32 -> 33).
constexpr int kMx4PairLeast = 128;  // rows, of an expert on average
constexpr int kMx4PairMore = 3;     // row tiles tried beyond the fewest

// A wave of pair tiles takes 0.19 us + 0.55 ns a row for every block and 0.3 us + 6 ns a
// row beside them, 5 us go before and after: fitted to 15 shapes (M 512 .. 4096) in
// tiles of 96 to 256 rows, of which it finds the fastest or one within 5 %.
double mx4_pair_cost(int n, int64_t tiles, int kblocks, double weight_bytes, int sms) {
  const double waves = static_cast<double>((tiles + sms / 2 - 1) / (sms / 2));
  const double t = 5.0 + waves * (kblocks * (0.19 + 0.00055 * n) + 0.3 + 0.006 * n);
  return std::max(t, 5.0 + weight_bytes / 5.5e6) + 0.05 * t;
}

bool mx4_experts_in_pairs(int64_t E, int64_t T, double flops) {
  return T >= kMx4PairLeast * E && flops * std::min<int64_t>(T / E, 256) >= 1.28e13;
}

// The row tiles of pairs at most for T rows or fewer.
int64_t mx4_pair_tiles(int64_t E, int64_t T, bool ragged) {
  if (T < kMx4PairLeast * (ragged ? E : 1)) return 0;
  return ragged ? E + T / kMx4PairLeast : (T + kMx4PairRows - 1) / kMx4PairRows + kMx4PairMore;
}

// ask: `sms` are the current device's, which says how many clusters it holds.
spense_status search_mx4_plan(int64_t E, int n_tiles, int kblocks, int64_t T, bool ragged, int sms, bool ask,
                              Mx4GemmPlan* out) {
  Mx4GemmPlan pl{};
  const uint32_t tail = static_cast<uint32_t>(round_up(kMx4BarrierBytes + 4 * (3 * static_cast<size_t>(E) + 1), 16));
  const int64_t active = ragged ? std::min(E, T) : 1;
  const double flops = 2.0 * T * n_tiles * kMx4Rows * kblocks * kMx4Cols;
  const int64_t avg = (T + E - 1) / E;
  pl.pair = ragged && mx4_experts_in_pairs(E, T, flops) ? 1 : 0;
  const int step = pl.pair ? 32 : 16;
  // Row tiles at most: every expert's last one may be short.
  auto row_tiles = [&](int n) { return ragged ? active + T / n : (T + n - 1) / n; };
  auto stage = [&](int n) {
    return kMx4BlockBytes + static_cast<uint32_t>(pl.pair ? n / 2 : n) * 128u + (pl.pair ? kMx4XsTileBytes : 0u);
  };
  auto slot = [&](int n) { return pl.pair ? 0u : (n > 61 ? 2048u : 1024u); };
  auto ring = [&](int n) {
    const uint32_t fixed = 1024 + tail + kMx4XsSlots * slot(n);
    return static_cast<int>(std::min<uint32_t>(12, (kMx4Smem - fixed) / stage(n)));
  };
  pl.split = 1;
  const double weight_bytes = static_cast<double>(active) * n_tiles * kblocks * kMx4BlockBytes;
  const int64_t m0 = ragged ? 1 : (T + kMx4MaxTile - 1) / kMx4MaxTile;
  double best = 0.0;
  for (int64_t m = m0; m < m0 + (ragged ? 1 : 16); ++m) {
    int n;
    if (ragged)
      n = pl.pair ? (avg >= 256 ? kMx4PairRows : 192)
                  : static_cast<int>(std::min<int64_t>(round_up(std::max<int64_t>(2 * avg, 32), 16), 208));
    else
      n = static_cast<int>(round_up((T + m - 1) / m, step));
    n = static_cast<int>(std::min<int64_t>(n, round_up(T, step)));
    const int64_t tiles = row_tiles(n) * n_tiles;
    for (int s = 1; s <= (pl.pair ? 1 : 8); ++s) {
      if (s > 1) {
        if (tiles * s > sms || kblocks < 2 * s || ring(n) < 3) break;
        const size_t partials = static_cast<size_t>(s - 1) * round_up((n + s - 1) / s, 8) * 512;
        if (partials > static_cast<size_t>(ring(n)) * stage(n) || tiles > clusters_at_once(s, sms, ask)) continue;
      }
      const double c = mx4_cost(n, s, tiles, kblocks, weight_bytes, sms);
      if (best == 0.0 || c < best) {
        best = c;
        pl.npad = n;
        pl.split = s;
      }
    }
    if (n <= step) break;
  }
  if (!ragged && T >= kMx4PairLeast) {
    // A CTA's later tiles also wait for the epilogues of the ones before.
    const int64_t singles = row_tiles(pl.npad) * n_tiles;
    if (pl.split == 1) best += 0.01 * pl.npad * static_cast<double>((singles + sms - 1) / sms - 1);
    const int64_t p0 = (T + kMx4PairRows - 1) / kMx4PairRows;
    for (int64_t m = p0; m <= p0 + kMx4PairMore; ++m) {
      const int n = static_cast<int>(round_up((T + m - 1) / m, 32));
      const double c = mx4_pair_cost(n, row_tiles(n) * ((n_tiles + 1) / 2), kblocks, weight_bytes, sms);
      if (c < best) {
        best = c;
        pl.pair = pl.split = 1;
        pl.npad = n;
      }
    }
  }
  pl.row_tiles = row_tiles(pl.npad);
  const int64_t tiles = pl.row_tiles * (pl.pair ? (n_tiles + 1) / 2 : n_tiles);
  if (tiles > INT_MAX / 8) return fail(SPENSE_ERR_SHAPE, "too many tiles for one launch (%lld)", (long long)tiles);
  pl.grid = static_cast<int>(pl.pair        ? 2 * std::min<int64_t>(tiles, sms / 2)
                             : pl.split > 1 ? tiles * pl.split
                                            : std::min<int64_t>(tiles, sms));
  pl.stage_bytes = stage(pl.npad);
  pl.xs_bytes = slot(pl.npad);
  pl.stages = ring(pl.npad);
  // Tensor memory: two accumulators where a CTA has several tiles, and 16 or 24
  // scale columns a block in the ring.
  const int sf_cols = pl.npad > 128 ? 24 : 16;
  pl.nacc = pl.split == 1 && 2 * pl.npad + 4 * sf_cols <= 512 ? 2 : 1;
  pl.stages = std::min(pl.stages, (512 - pl.nacc * pl.npad) / sf_cols);
  // Small tiles: two blocks a stage, which halves the waits and signals a block costs
  // the issuing warp (10240x5120 at one row 8.7 -> 7.5 us in the run that compared
  // them, 64-expert decode 37.9 -> 36.2 us; with more than 64 rows the products cover
  // them: the same either way).
  pl.bps = 1;
  if (!pl.pair && pl.npad <= 64 && pl.stages >= 6) {
    pl.bps = 2;
    pl.stages /= 2;
    pl.stage_bytes *= 2;
    pl.xs_bytes *= 2;
  }
  if (pl.stages < 3) return fail(SPENSE_ERR_SHAPE, "no launch plan for %lld experts", (long long)E);
  pl.tmem_cols = 32;
  while (pl.tmem_cols < static_cast<uint32_t>(pl.nacc * pl.npad + pl.stages * pl.bps * sf_cols)) pl.tmem_cols <<= 1;
  pl.smem_bytes = 1024 + tail + kMx4XsSlots / pl.bps * pl.xs_bytes + static_cast<uint32_t>(pl.stages) * pl.stage_bytes;
  pl.workspace_bytes = kMx4Header + (pl.pair ? static_cast<size_t>(pl.row_tiles) * kblocks * kMx4XsTileBytes : 0);
  *out = pl;
  return SPENSE_OK;
}

// The search takes some 3 us; a thread keeps the plans of its last shapes.
spense_status make_mx4_plan(int64_t E, int n_tiles, int kblocks, int64_t T, bool ragged, int sms, Mx4GemmPlan* out) {
  struct Known {
    std::array<int64_t, 6> key{};
    Mx4GemmPlan plan{};
  };
  static thread_local std::array<Known, 64> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  const std::array<int64_t, 6> key = {E, n_tiles, kblocks, T, (ragged ? 1 : 2) + 4 * (dev + 1), sms};
  uint64_t h = 0;
  for (const int64_t k : key) h = (h ^ static_cast<uint64_t>(k)) * 0x9E3779B97F4A7C15ull;
  Known& slot = known[h >> 58];
  if (slot.key != key) {
    const spense_status st = search_mx4_plan(E, n_tiles, kblocks, T, ragged, sms, true, &slot.plan);
    if (st != SPENSE_OK) {
      slot.key = {};
      return st;
    }
    slot.key = key;
  }
  *out = slot.plan;
  return SPENSE_OK;
}

spense_status check_mx4_types(int64_t rows, int64_t K) {
  if (rows < 0 || rows > kMx4MaxRows)
    return fail(SPENSE_ERR_SHAPE, "%lld rows outside [0, 2^20]", (long long)rows);
  if (K < 32 || K > (1 << 20) || K % 32 != 0)
    return fail(SPENSE_ERR_SHAPE, "K = %lld must be a multiple of 32 in [32, 2^20]", (long long)K);
  return SPENSE_OK;
}

// The activation scales' words of a product's rows are counted in 32 bits.
spense_status check_mx4_words(int64_t rows, int64_t K) {
  const int64_t words = (K + 127) / 128 * rows;
  if (words > INT_MAX)
    return fail(SPENSE_ERR_SHAPE, "%lld words of activation scales (%lld rows of K = %lld), at most 2^31 - 1",
                (long long)words, (long long)rows, (long long)K);
  return SPENSE_OK;
}

// A packed weight's shape; its 128-row tiles and 256-column blocks.
spense_status check_mx4_weight(int64_t E, int64_t N, int64_t K, int64_t* n_tiles, int64_t* kblocks) {
  if (E < 1 || E > kMx4MaxExperts)
    return fail(SPENSE_ERR_SHAPE, "%lld experts outside [1, %d]", (long long)E, kMx4MaxExperts);
  if (N < 1 || N > (1 << 20)) return fail(SPENSE_ERR_SHAPE, "N = %lld outside [1, 2^20]", (long long)N);
  const spense_status st = check_mx4_types(0, K);
  if (st != SPENSE_OK) return st;
  *n_tiles = (N + kMx4Rows - 1) / kMx4Rows;
  *kblocks = (K + kMx4Cols - 1) / kMx4Cols;
  if (E * *n_tiles * *kblocks > INT_MAX / (kMx4BlockBytes / 128))
    return fail(SPENSE_ERR_SHAPE, "too many blocks for one weight (%lld)", (long long)(E * *n_tiles * *kblocks));
  return SPENSE_OK;
}

spense_status run_mx4(const spense_mx4_packed* h, const uint8_t* Xq, const uint8_t* x_scale, int64_t T,
                      const int32_t* offsets, uint16_t* Y, int64_t ldy, void* workspace, size_t workspace_bytes,
                      void* stream) {
  if (h == nullptr) return fail(SPENSE_ERR_ARG, "Wp is NULL");
  if (T < 0 || T > kMx4MaxRows) return fail(SPENSE_ERR_SHAPE, "%lld rows outside [0, 2^20]", (long long)T);
  spense_status st = check_mx4_words(T, h->K);
  if (st != SPENSE_OK) return st;
  if (T > 0 && (Xq == nullptr || x_scale == nullptr || Y == nullptr))
    return fail(SPENSE_ERR_ARG, "Xq, x_scale or Y is NULL");
  if (ldy < h->N || ldy > (1 << 30))
    return fail(SPENSE_ERR_SHAPE, "ldy = %lld outside [N = %lld, 2^30]", (long long)ldy, (long long)h->N);
  if (!aligned(Xq, 16) || !aligned(x_scale, 16) || !aligned(Y, 16))
    return fail(SPENSE_ERR_ALIGN, "Xq, x_scale and Y must be 16-byte aligned");
  if (workspace == nullptr) return fail(SPENSE_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(workspace, 256)) return fail(SPENSE_ERR_ALIGN, "workspace is not 256-byte aligned");
  int dev = 0;
  DeviceInfo info;
  st = current_device(&dev, &info);
  if (st != SPENSE_OK) return st;
  if (dev != h->device)
    return fail(SPENSE_ERR_ARG, "handle was packed on device %d, current device is %d", h->device, dev);
  if (T == 0) return ok();
  Mx4GemmPlan pl;
  st = make_mx4_plan(h->E, h->n_tiles, h->kblocks, T, offsets != nullptr, info.sms, &pl);
  if (st != SPENSE_OK) return st;
  if (workspace_bytes < pl.workspace_bytes)
    return fail(SPENSE_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", workspace_bytes, pl.workspace_bytes);
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return fail(SPENSE_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  Mx4GemmParams p{};
  Mx4GemmMaps maps;
  for (int i = 0; i < 3; ++i) {
    p.box[i] = std::min(pl.pair ? pl.npad / 2 : pl.npad, i == 0 ? 16 : (i == 1 ? 64 : 256));
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(h->K / 2), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(h->K / 2)};
    const cuuint32_t box[2] = {128u, static_cast<cuuint32_t>(p.box[i])};
    const cuuint32_t estr[2] = {1u, 1u};
    const CUresult r = encode(&maps.x[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(Xq), dims, strides,
                              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SPENSE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  }
  const int64_t groups = (h->K + 127) / 128;
  for (int i = 0; i < 2; ++i) {
    const cuuint64_t dims[1] = {static_cast<cuuint64_t>(groups * T)};
    const cuuint64_t strides[1] = {0};  // a one-dimensional map has none
    const cuuint32_t box[1] = {i == 0 ? 64u : 256u}, estr[1] = {1u};
    const CUresult r = encode(i == 0 ? &maps.xs_narrow : &maps.xs_wide, CU_TENSOR_MAP_DATA_TYPE_UINT32, 1,
                              const_cast<uint8_t*>(x_scale), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SPENSE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  }
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  for (int i = 0; pl.pair && i < 2; ++i) {
    const uint32_t rows = (i == 0 ? kMx4BlockBytes : kMx4XsTileBytes) / 128;
    const cuuint64_t blocks = (i == 0 ? static_cast<cuuint64_t>(h->E) * h->n_tiles : pl.row_tiles) * h->kblocks;
    const cuuint64_t dims[2] = {32, blocks * rows};
    const cuuint64_t strides[1] = {128};
    const cuuint32_t box[2] = {32u, rows}, estr[2] = {1u, 1u};
    const CUresult r = encode(i == 0 ? &maps.w : &maps.xs_tiles, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2,
                              i == 0 ? h->blocks : ws + kMx4Header, dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SPENSE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  }
  p.blocks = h->blocks;
  p.xs = reinterpret_cast<const uint32_t*>(x_scale);
  p.y = Y;
  p.ldy = ldy;
  p.offsets = offsets;
  p.status = reinterpret_cast<unsigned int*>(ws);
  p.test_gate = nullptr;
#ifdef SPENSE_TEST_HOOKS
  // Test build only: with SPENSE_TEST_STALL=1 the loaders wait on header word
  // 16 of the workspace, which nothing sets, so every launch ends by timeout.
  static const bool stall = std::getenv("SPENSE_TEST_STALL") != nullptr && std::getenv("SPENSE_TEST_STALL")[0] == '1';
  if (stall) p.test_gate = reinterpret_cast<const unsigned int*>(ws + 64);
#endif
  p.E = static_cast<int>(h->E);
  p.N = static_cast<int>(h->N);
  p.T = static_cast<int>(T);
  p.n_tiles = h->n_tiles;
  p.kblocks = h->kblocks;
  p.groups = static_cast<int>(groups);
  const int tail_cols = static_cast<int>(h->K - static_cast<int64_t>(h->kblocks - 1) * kMx4Cols);
  p.last_steps = (tail_cols + 63) / 64;
  p.npad = pl.npad;
  // Activation codes of up to 32 MB stay in L2 while all weights pass, and the weights
  // are read once. More of them go in groups of 24 row tiles: 5120x27648 at 16384 rows
  // 1051 -> 901 us (in groups of 12 950, of 32 953), 20480x5120 at 32768 rows 1377 ->
  // 1350 (of 12 1527, of 16 1383).
  p.group = T * (h->K / 2) <= (32 << 20) ? 1 << 16 : 24;
  p.stages = pl.stages;
  p.nacc = pl.nacc;
  p.bps = pl.bps;
  p.split = pl.split;
  p.pair = pl.pair;
  p.stage_bytes = pl.stage_bytes;
  p.xs_bytes = pl.xs_bytes;
  p.tmem_cols = pl.tmem_cols;
  p.w_keep = T > pl.npad ? 1 : 0;
  cudaError_t e = cudaSuccess;
  if (pl.pair)
    e = launch_mx4_scale_tiles(p, static_cast<int>(pl.row_tiles), reinterpret_cast<uint32_t*>(ws + kMx4Header),
                               static_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = launch_mx4_gemm(maps, p, pl.grid, pl.smem_bytes, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "mx4 gemm launch");
  return ok();
}

}  // namespace

extern "C" {

spense_status spense_mx4_quantize(const void* X, int x_type, int64_t M, int64_t K, int64_t ldx, const int32_t* rows,
                                  int64_t T, uint8_t* Xq, uint8_t* x_scale, unsigned int flags, void* stream) {
  if (x_type != SPENSE_TYPE_BF16 && x_type != SPENSE_TYPE_F16 && x_type != SPENSE_TYPE_F32)
    return fail(SPENSE_ERR_ARG, "unknown x_type %d", x_type);
  if (flags & ~static_cast<unsigned int>(SPENSE_MX4_SCALE_ROWS))
    return fail(SPENSE_ERR_ARG, "unknown flags 0x%x", flags);
  spense_status st = check_mx4_types(M, K);
  if (st != SPENSE_OK) return st;
  st = check_mx4_types(T, K);
  if (st != SPENSE_OK) return st;
  if (rows == nullptr && T != M)
    return fail(SPENSE_ERR_SHAPE, "T = %lld must equal M = %lld without rows", (long long)T, (long long)M);
  if (ldx < K || ldx > (1 << 30))
    return fail(SPENSE_ERR_SHAPE, "ldx = %lld outside [K = %lld, 2^30]", (long long)ldx, (long long)K);
  if (T > 0 && (Xq == nullptr || x_scale == nullptr || (M > 0 && X == nullptr)))
    return fail(SPENSE_ERR_ARG, "X, Xq or x_scale is NULL");
  const int64_t esize = x_type == SPENSE_TYPE_F32 ? 4 : 2;
  if (!aligned(X, 16) || !aligned(Xq, 16) || !aligned(x_scale, 16) || !aligned(rows, 4) || (ldx * esize) % 16 != 0)
    return fail(SPENSE_ERR_ALIGN, "X (and each of its rows), Xq and x_scale must be 16-byte aligned, rows 4-byte");
  int dev = 0;
  DeviceInfo info;
  st = current_device(&dev, &info);
  if (st != SPENSE_OK) return st;
  const cudaError_t e = launch_mx4_quantize(X, x_type, T, K, ldx, rows, M, Xq, x_scale,
                                            (flags & SPENSE_MX4_SCALE_ROWS) == 0, info.sms,
                                            static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "mx4 quantize launch");
  return ok();
}

spense_status spense_mx4_dequantize(const uint8_t* Xq, const uint8_t* x_scale, int64_t M, int64_t K, void* Y,
                                    int y_type, unsigned int flags, void* stream) {
  if (y_type != SPENSE_TYPE_BF16 && y_type != SPENSE_TYPE_F32) return fail(SPENSE_ERR_ARG, "unknown y_type %d", y_type);
  if (flags & ~static_cast<unsigned int>(SPENSE_MX4_SCALE_ROWS))
    return fail(SPENSE_ERR_ARG, "unknown flags 0x%x", flags);
  spense_status st = check_mx4_types(M, K);
  if (st != SPENSE_OK) return st;
  if (M > 0 && (Xq == nullptr || x_scale == nullptr || Y == nullptr))
    return fail(SPENSE_ERR_ARG, "Xq, x_scale or Y is NULL");
  if (!aligned(Xq, 16) || !aligned(x_scale, 16) || !aligned(Y, 16))
    return fail(SPENSE_ERR_ALIGN, "Xq, x_scale and Y must be 16-byte aligned");
  int dev = 0;
  DeviceInfo info;
  st = current_device(&dev, &info);
  if (st != SPENSE_OK) return st;
  const cudaError_t e = launch_mx4_dequantize(Xq, x_scale, (flags & SPENSE_MX4_SCALE_ROWS) == 0, M, K, Y, y_type,
                                              info.sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "mx4 dequantize launch");
  return ok();
}

spense_status spense_mx4_pack(const uint8_t* Wq, const uint8_t* w_scale, int64_t E, int64_t N, int64_t K,
                              void* stream_v, spense_mx4_packed** out) {
  if (out == nullptr) return fail(SPENSE_ERR_ARG, "out is NULL");
  *out = nullptr;
  if (Wq == nullptr || w_scale == nullptr) return fail(SPENSE_ERR_ARG, "Wq or w_scale is NULL");
  int64_t n_tiles = 0, kblocks = 0;
  spense_status st = check_mx4_weight(E, N, K, &n_tiles, &kblocks);
  if (st != SPENSE_OK) return st;
  if (!aligned(Wq, 16)) return fail(SPENSE_ERR_ALIGN, "Wq is not 16-byte aligned");
  int dev = 0;
  DeviceInfo info;
  st = current_device(&dev, &info);
  if (st != SPENSE_OK) return st;
  spense_mx4_packed* h = new (std::nothrow) spense_mx4_packed;
  if (h == nullptr) return fail(SPENSE_ERR_OOM, "out of host memory");
  h->device = dev;
  h->E = E;
  h->N = N;
  h->K = K;
  h->n_tiles = static_cast<int>(n_tiles);
  h->kblocks = static_cast<int>(kblocks);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
  unsigned int* err_d = nullptr;
  unsigned int err = 0;
  cudaError_t e = cudaMalloc(reinterpret_cast<void**>(&h->blocks),
                             static_cast<size_t>(E * n_tiles * kblocks) * kMx4BlockBytes);
  if (e == cudaSuccess) e = cudaMalloc(reinterpret_cast<void**>(&err_d), sizeof(unsigned int));
  if (e == cudaSuccess) e = cudaMemsetAsync(err_d, 0, sizeof(unsigned int), stream);
  if (e == cudaSuccess)
    e = launch_mx4_pack(Wq, w_scale, E, N, K, h->n_tiles, h->kblocks, h->blocks, err_d, stream);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&err, err_d, sizeof(err), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (err_d != nullptr) cudaFree(err_d);
  if (e != cudaSuccess || err != 0) {
    spense_mx4_free(h);
    if (e != cudaSuccess) return cuda_fail(e, "mx4 pack");
    return fail(SPENSE_ERR_NONFINITE, "w_scale holds a NaN byte (255)");
  }
  *out = h;
  return ok();
}

spense_status spense_mx4_free(spense_mx4_packed* Wp) {
  if (Wp != nullptr) {
    if (Wp->blocks != nullptr) cudaFree(Wp->blocks);
    delete Wp;
  }
  return ok();
}

spense_status spense_mx4_get_info(const spense_mx4_packed* Wp, spense_mx4_info* info) {
  if (Wp == nullptr || info == nullptr) return fail(SPENSE_ERR_ARG, "NULL argument");
  info->E = Wp->E;
  info->N = Wp->N;
  info->K = Wp->K;
  info->n_tiles = Wp->n_tiles;
  info->k_blocks = Wp->kblocks;
  info->blocks = Wp->blocks;
  info->weight_bytes = static_cast<uint64_t>(Wp->E) * Wp->n_tiles * Wp->kblocks * kMx4BlockBytes;
  return ok();
}

size_t spense_mx4_workspace_size(const spense_mx4_packed* Wp, int64_t M) {
  if (Wp == nullptr || M < 0 || M > kMx4MaxRows) {
    fail(SPENSE_ERR_ARG, "Wp is NULL or M outside [0, 2^20]");
    return 0;
  }
  if (check_mx4_words(M, Wp->K) != SPENSE_OK) return 0;
  // A weight of one expert serves both products, which may be planned differently.
  // Enough for fewer rows too, whose tiles may be more.
  int64_t tiles = mx4_pair_tiles(Wp->E, M, true);
  if (Wp->E == 1) tiles = std::max(tiles, mx4_pair_tiles(1, M, false));
  return kMx4Header + static_cast<size_t>(tiles) * Wp->kblocks * kMx4XsTileBytes;
}

spense_status spense_mx4_plan_shapes(int64_t E, int64_t N, int64_t K, int64_t M, int grouped, int sms,
                                     spense_mx4_plan_info* out) {
  if (out == nullptr) return fail(SPENSE_ERR_ARG, "out is NULL");
  if (sms < 1 || sms > 1024) return fail(SPENSE_ERR_ARG, "sms = %d outside [1, 1024]", sms);
  if (E != 1 && !grouped) return fail(SPENSE_ERR_ARG, "%lld experts without grouped", (long long)E);
  int64_t n_tiles = 0, kblocks = 0;
  spense_status st = check_mx4_weight(E, N, K, &n_tiles, &kblocks);
  if (st == SPENSE_OK) st = check_mx4_types(M, K);
  if (st == SPENSE_OK) st = check_mx4_words(M, K);
  if (st != SPENSE_OK) return st;
  if (M == 0) return fail(SPENSE_ERR_SHAPE, "no rows, no launch");
  int dev = 0, device_sms = 0;
  const bool ask = cudaGetDevice(&dev) == cudaSuccess &&
                   cudaDeviceGetAttribute(&device_sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
                   device_sms == sms;
  if (!ask) cudaGetLastError();
  Mx4GemmPlan pl;
  st = search_mx4_plan(E, static_cast<int>(n_tiles), static_cast<int>(kblocks), M, grouped != 0, sms, ask, &pl);
  if (st != SPENSE_OK) return st;
  *out = spense_mx4_plan_info{};
  out->npad = pl.npad;
  out->pair = pl.pair;
  out->split = pl.split;
  out->grid = pl.grid;
  out->stages = pl.stages;
  out->blocks_per_stage = pl.bps;
  out->nacc = pl.nacc;
  out->tmem_cols = pl.tmem_cols;
  out->smem_bytes = pl.smem_bytes;
  out->stage_bytes = pl.stage_bytes;
  out->n_tiles = n_tiles;
  out->k_blocks = kblocks;
  out->row_tiles = pl.row_tiles;
  out->workspace_bytes = pl.workspace_bytes;
  return ok();
}

spense_status spense_mx4_gemm(const spense_mx4_packed* Wp, const uint8_t* Xq, const uint8_t* x_scale, int64_t M,
                              uint16_t* Y, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  if (Wp != nullptr && Wp->E != 1)
    return fail(SPENSE_ERR_ARG, "the weight holds %lld experts: use spense_mx4_gemm_experts", (long long)Wp->E);
  return run_mx4(Wp, Xq, x_scale, M, nullptr, Y, ldy, workspace, workspace_bytes, stream);
}

spense_status spense_mx4_gemm_experts(const spense_mx4_packed* Wp, const uint8_t* Xq, const uint8_t* x_scale,
                                      int64_t T, const int32_t* offsets, uint16_t* Y, int64_t ldy, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  if (offsets == nullptr) return fail(SPENSE_ERR_ARG, "offsets is NULL");
  if (!aligned(offsets, 4)) return fail(SPENSE_ERR_ALIGN, "offsets is not 4-byte aligned");
  return run_mx4(Wp, Xq, x_scale, T, offsets, Y, ldy, workspace, workspace_bytes, stream);
}

size_t spense_expert_sort_workspace_size(int64_t M, int64_t k, int64_t E) {
  if (M < 0 || M > kMx4MaxRows || k < 1 || k > 64 || M * k > (1 << 24) || E < 1 || E > kMx4MaxExperts) {
    fail(SPENSE_ERR_SHAPE, "M = %lld, k = %lld or E = %lld out of range", (long long)M, (long long)k, (long long)E);
    return 0;
  }
  return round_up(static_cast<size_t>(expert_sort_counts(M * k, E)) * 4, 256);
}

spense_status spense_expert_sort(const void* ids, int id_bits, int64_t M, int64_t k, int64_t E, int32_t* offsets,
                                 int32_t* rows, int32_t* pos, void* workspace, size_t workspace_bytes, void* stream) {
  if (id_bits != 32 && id_bits != 64) return fail(SPENSE_ERR_ARG, "id_bits is %d, not 32 or 64", id_bits);
  const size_t need = spense_expert_sort_workspace_size(M, k, E);
  if (need == 0) return SPENSE_ERR_SHAPE;
  if (offsets == nullptr || (M > 0 && (ids == nullptr || rows == nullptr || pos == nullptr)))
    return fail(SPENSE_ERR_ARG, "ids, offsets, rows or pos is NULL");
  if (!aligned(ids, id_bits / 8) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4))
    return fail(SPENSE_ERR_ALIGN, "ids, offsets, rows and pos must be aligned to their type");
  if (workspace == nullptr) return fail(SPENSE_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(workspace, 256)) return fail(SPENSE_ERR_ALIGN, "workspace is not 256-byte aligned");
  if (workspace_bytes < need)
    return fail(SPENSE_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", workspace_bytes, need);
  int dev = 0;
  DeviceInfo info;
  const spense_status st = current_device(&dev, &info);
  if (st != SPENSE_OK) return st;
  const cudaError_t e = launch_expert_sort(ids, id_bits == 64, M * k, static_cast<int>(k), static_cast<int>(E),
                                           offsets, rows, pos, static_cast<int32_t*>(workspace),
                                           static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "expert sort launch");
  return ok();
}

spense_status spense_expert_combine(const uint16_t* Y, int64_t T, int64_t N, int64_t ldy, const int32_t* pos,
                                    const float* weights, int64_t M, int64_t k, uint16_t* out, int64_t ldo,
                                    void* stream) {
  if (T < 0 || T > (1 << 24) || M < 0 || M > kMx4MaxRows || k < 1 || k > 64 || N < 1 || N > (1 << 20))
    return fail(SPENSE_ERR_SHAPE, "T = %lld, M = %lld, k = %lld or N = %lld out of range", (long long)T, (long long)M,
                (long long)k, (long long)N);
  if (ldy < N || ldy > (1 << 30) || ldo < N || ldo > (1 << 30))
    return fail(SPENSE_ERR_SHAPE, "ldy = %lld or ldo = %lld outside [N = %lld, 2^30]", (long long)ldy, (long long)ldo,
                (long long)N);
  if (M > 0 && ((T > 0 && Y == nullptr) || pos == nullptr || weights == nullptr || out == nullptr))
    return fail(SPENSE_ERR_ARG, "Y, pos, weights or out is NULL");
  if (!aligned(Y, 16) || !aligned(out, 16) || !aligned(pos, 4) || !aligned(weights, 4))
    return fail(SPENSE_ERR_ALIGN, "Y and out must be 16-byte aligned, pos and weights 4-byte");
  int dev = 0;
  DeviceInfo info;
  const spense_status st = current_device(&dev, &info);
  if (st != SPENSE_OK) return st;
  const cudaError_t e = launch_expert_combine(Y, T, N, ldy, pos, weights, M, static_cast<int>(k), out, ldo,
                                              static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "expert combine launch");
  return ok();
}

}  // extern "C"
