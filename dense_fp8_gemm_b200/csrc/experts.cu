// The rows of a mixture of experts: the stable sort of every token's choices
// by expert, in front of the products grouped by expert, and the weighted sum of
// each token's rows behind them.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>

#include "mx4_internal.h"
#include "pdl.cuh"

namespace spense {
namespace {

// ---------------------------------------------------------------- sort
// A counting sort: position of choice i = (choices of smaller experts) +
// (earlier choices of the same expert). The choices are cut into chunks of one
// CTA each, and a chunk into 32 contiguous runs of one warp each; a warp takes
// its run 32 choices at a time and finds the equal ones among them by ballots, so
// nothing depends on the order in which warps or CTAs arrive and the result is the
// stable one.
//   kSingle  the one chunk: counts, offsets and positions in one launch.
//   kCount   counts of a chunk into counts[E][chunks].
//   kPlace   recounts the chunk and takes its bases from all chunks' counts, a
//            warp an expert at a time, so that they are read in whole lines (one
//            thread an expert took 18.4 us for 131072 choices of 256 experts).
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kKept = 4;  // rounds of 32 choices a warp keeps in registers
enum SortMode { kSingle, kCount, kPlace };

template <bool kWide>
__device__ __forceinline__ int expert_of(const void* ids, int i, int end, int E) {
  if (i >= end) return E;
  if constexpr (kWide) {
    const long long v = ld_dep(static_cast<const long long*>(ids) + i);
    return v >= 0 && v < E ? static_cast<int>(v) : E;
  } else {
    const int v = ld_dep(static_cast<const int*>(ids) + i);
    return v >= 0 && v < E ? v : E;
  }
}

// Lanes with the same expert, by its bits: one ballot each. (The match instruction
// goes through the different values one by one: 4096 choices of 128 experts took
// 11.7 us with it.)
__device__ __forceinline__ uint32_t lanes_with(int e, int bits) {
  uint32_t same = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const bool set = (e >> b) & 1;
    const uint32_t v = __ballot_sync(0xffffffffu, set);
    same &= set ? v : ~v;
  }
  return same;
}

template <bool kWide, SortMode kMode>
__global__ void __launch_bounds__(kSortThreads)
    expert_sort_kernel(const void* ids, int n, int k, int E, int bits, int chunk,
                       int32_t* __restrict__ offsets,
                       int32_t* __restrict__ rows, int32_t* __restrict__ pos, int32_t* counts) {
  extern __shared__ int hist[];  // [warps][E]: the warp's choices of an expert, then its first position
  __shared__ int warp_sum[kSortWarps];
  __shared__ int total_live;
  const int stride = (gridDim.x + 3) & ~3;  // of counts, so that four are 16 bytes
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
  pdl_trigger();
  for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  pdl_wait();
  const int c0 = blockIdx.x * chunk, c1 = min(n, c0 + chunk);
  const int run = ((chunk + kSortThreads - 1) / kSortThreads) * 32;
  const int i0 = min(c1, c0 + warp * run), i1 = min(c1, i0 + run);
  int* const mine = hist + warp * E;
  // The run's first kKept rounds stay in registers for the second pass.
  int kept[kKept];
  uint32_t kept_same[kKept];
#pragma unroll
  for (int q = 0; q < kKept; ++q) kept[q] = expert_of<kWide>(ids, i0 + 32 * q + lane, i1, E);
#pragma unroll
  for (int q = 0; q < kKept; ++q) kept_same[q] = i0 + 32 * q < i1 ? lanes_with(kept[q], bits) : 0u;
  auto count = [&](int e, uint32_t same) {
    if (e < E && (same & below) == 0u) mine[e] += __popc(same);
    __syncwarp();
  };
#pragma unroll
  for (int q = 0; q < kKept; ++q)
    if (i0 + 32 * q < i1) count(kept[q], kept_same[q]);
  for (int b = i0 + 32 * kKept; b < i1; b += 32) {
    const int e = expert_of<kWide>(ids, b + lane, i1, E);
    count(e, lanes_with(e, bits));
  }
  __syncthreads();
  // Thread t: the expert t (E <= 1024). Its choices in this chunk, and before it.
  const int t = threadIdx.x;
  const int warps = min(kSortWarps, (c1 - c0 + run - 1) / run);  // with choices
  int sum = 0, before = 0;
  if (t < E) {
    for (int w0 = 0; w0 < warps; w0 += 8) {  // eight reads in flight (a warp without choices counted none)
      int c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = hist[(w0 + w) * E + t];
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        hist[(w0 + w) * E + t] = sum;
        sum += c[w];
      }
    }
  }
  if constexpr (kMode == kCount) {
    if (t < E) counts[t * stride + blockIdx.x] = sum;
    return;
  }
  int total = sum;
  if constexpr (kMode == kPlace) {
    __shared__ int2 bases[kMx4MaxExperts];
    // A lane takes four chunks' counts (there are 128 chunks at most), a warp four
    // experts at a time.
    const int chunks = static_cast<int>(gridDim.x), c = 4 * lane;
    for (int e0 = warp; e0 < E; e0 += 4 * kSortWarps) {
      int4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = e0 + u * kSortWarps;
        v[u] = make_int4(0, 0, 0, 0);
        if (e < E && c < chunks) v[u] = ld_dep(reinterpret_cast<const int4*>(counts + e * stride + c));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = e0 + u * kSortWarps;
        const int w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        int all = 0, less = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          all += c + q < chunks ? w[q] : 0;
          less += c + q < static_cast<int>(blockIdx.x) ? w[q] : 0;
        }
        all = __reduce_add_sync(0xffffffffu, all);
        less = __reduce_add_sync(0xffffffffu, less);
        if (lane == 0 && e < E) bases[e] = make_int2(all, less);
      }
    }
    __syncthreads();
    if (t < E) {
      total = bases[t].x;
      before = bases[t].y;
    }
  }
  // Exclusive scan of the experts' totals: the offsets.
  int scan = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) warp_sum[warp] = scan;
  __syncthreads();
  if (warp == 0) {
    int v = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    warp_sum[lane] = v;
    if (lane == 31) total_live = v;
  }
  __syncthreads();
  const int first = scan - total + (warp > 0 ? warp_sum[warp - 1] : 0);
  if (t < E) {
    if (blockIdx.x == 0) offsets[t] = first;
    for (int w0 = 0; w0 < warps; w0 += 8) {
      int c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = hist[(w0 + w) * E + t];
#pragma unroll
      for (int w = 0; w < 8; ++w) hist[(w0 + w) * E + t] = c[w] + first + before;
    }
  }
  if (blockIdx.x == 0 && t == 0) offsets[E] = total_live;
  __syncthreads();
  auto place = [&](int i, int e, uint32_t same) {
    const uint32_t earlier = same & below;
    int p = -1;
    if (e < E) p = mine[e] + __popc(earlier);
    __syncwarp();
    if (e < E && earlier == 0u) mine[e] += __popc(same);
    __syncwarp();
    if (i < i1) {
      pos[i] = p;
      if (p >= 0) rows[p] = static_cast<int>(static_cast<unsigned>(i) / static_cast<unsigned>(k));
    }
  };
#pragma unroll
  for (int q = 0; q < kKept; ++q)
    if (i0 + 32 * q < i1) place(i0 + 32 * q + lane, kept[q], kept_same[q]);
  for (int b = i0 + 32 * kKept; b < i1; b += 32) {
    const int e = expert_of<kWide>(ids, b + lane, i1, E);
    place(b + lane, e, lanes_with(e, bits));
  }
  // The slots behind the last expert's (as many as there are choices left out).
  for (int i = total_live + blockIdx.x * kSortThreads + t; i < n; i += gridDim.x * kSortThreads) rows[i] = -1;
}

// ---------------------------------------------------------------- combine
// out[m][n] = bf16(sum over j of weights[m][j] * Y[pos[m][j]][n]) in fp32, j
// ascending, choices with pos outside [0, T) left out (their weight is not
// looked at). Bound by the gathered rows' bytes: 8191 x 8 rows of 5120 columns in 116
// us, 6.5 TB/s or 0.99 of the measured copy rate, and 108 us (0.97) with a tenth of the
// choices dropped; under a load of seconds 120 and 115 us. The inputs are not __restrict__, so that they are
// read by plain (coherent) loads: the grid before may still have been writing them.
constexpr int kCombineThreads = 128;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Token and piece of thread or warp `i` where a token has `pieces` of them, in order.
__device__ __forceinline__ int64_t token_of(int64_t i, unsigned int pieces, unsigned int& piece) {
  const int64_t m = i >> 32 ? i / pieces : static_cast<unsigned int>(i) / pieces;
  piece = static_cast<unsigned int>(i - m * pieces);
  return m;
}

// Rows 16-byte aligned: eight columns a thread.
__global__ void __launch_bounds__(kCombineThreads)
    expert_combine_kernel(const uint16_t* Y, int64_t T, int64_t N, int64_t ldy,
                          const int32_t* pos, const float* weights, int64_t M, int k,
                          uint16_t* out, int64_t ldo) {
  pdl_trigger();
  unsigned int piece;
  const int64_t m = token_of(static_cast<int64_t>(blockIdx.x) * kCombineThreads + threadIdx.x,
                             static_cast<unsigned int>(N / 8), piece);
  const int64_t n = static_cast<int64_t>(piece) * 8;
  pdl_wait();
  if (m >= M) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  const int32_t* pm = pos + m * k;
  const float* wm = weights + m * k;
  for (int j0 = 0; j0 < k; j0 += 8) {
    float w[8];
    bool live[8];
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      live[j] = false;
      w[j] = 0.0f;
      v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (j0 + j < k) {
        const int64_t p = pm[j0 + j];
        live[j] = p >= 0 && p < T;
        if (live[j]) {
          w[j] = wm[j0 + j];
          v[j] = *reinterpret_cast<const uint4*>(Y + p * ldy + n);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!live[j]) continue;
      const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w[j], __uint_as_float(u[i] << 16), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w[j], __uint_as_float(u[i] & 0xFFFF0000u), acc[2 * i + 1]);
      }
    }
  }
  *reinterpret_cast<uint4*>(out + m * ldo + n) = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                                            pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
}

// Rows on any 2-byte boundary: a warp takes 512 columns of a token, lane l the
// pairs at 2 l, 64 + 2 l, .., so that every access is a word and a warp's are 128
// contiguous bytes. In a row that starts on an odd element a pair straddles two
// words: the second comes from the next lane. Nothing behind a row's last column is
// read (a pair that ends the row is read as single values). Eight pairs a lane and two
// rows at a time measured best: 5387 x 8 rows of 1307 columns 35 us (four pairs, four
// rows 44 us; eight neighbouring columns a thread 53 us), 9456 rows of 5065 54 us. Half
// of HBM's rate: 4-byte accesses instead of 16-byte ones bound it.
constexpr int kAnyPairs = 8, kAnyRows = 2;
__global__ void __launch_bounds__(kCombineThreads, 8)
    expert_combine_any_kernel(const uint16_t* Y, int64_t T, int64_t N, int64_t ldy,
                              const int32_t* pos, const float* weights, int64_t M, int k,
                              uint16_t* out, int64_t ldo) {
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  unsigned int window;
  const int64_t m = token_of(static_cast<int64_t>(blockIdx.x) * (kCombineThreads / 32) + (threadIdx.x >> 5),
                             static_cast<unsigned int>((N + 64 * kAnyPairs - 1) / (64 * kAnyPairs)), window);
  const int64_t n0 = static_cast<int64_t>(window) * 64 * kAnyPairs;
  pdl_wait();
  if (m >= M) return;  // the whole warp
  const int cols = static_cast<int>(N - n0 < 64 * kAnyPairs ? N - n0 : 64 * kAnyPairs);
  float lo[kAnyPairs], hi[kAnyPairs];
#pragma unroll
  for (int i = 0; i < kAnyPairs; ++i) lo[i] = hi[i] = 0.0f;
  const int32_t* pm = pos + m * k;
  const float* wm = weights + m * k;
  for (int j0 = 0; j0 < k; j0 += kAnyRows) {
    float w[kAnyRows];
    bool live[kAnyRows], odd[kAnyRows];
    uint32_t x[kAnyRows][kAnyPairs + 1];
#pragma unroll
    for (int j = 0; j < kAnyRows; ++j) {
      live[j] = odd[j] = false;
      w[j] = 0.0f;
      if (j0 + j >= k) continue;
      const int64_t p = pm[j0 + j];
      if (p < 0 || p >= T) continue;
      live[j] = true;
      w[j] = wm[j0 + j];
      const uint16_t* row = Y + p * ldy + n0;
      odd[j] = (reinterpret_cast<uintptr_t>(row) & 2) != 0;
      const uint32_t* words = reinterpret_cast<const uint32_t*>(row - (odd[j] ? 1 : 0));
#pragma unroll
      for (int i = 0; i <= kAnyPairs; ++i) {
        const int c = 64 * i + 2 * lane;  // the pair's first column
        x[j][i] = 0u;
        if (i == kAnyPairs && lane > 0) continue;  // behind a whole window's last pair, for lane 31
        if (c + 1 < cols || (odd[j] && c < cols))
          x[j][i] = words[32 * i + lane];
        else if (c < cols)
          x[j][i] = row[c];
        else if (odd[j] && c == cols)
          x[j][i] = row[c - 1];  // the last column: the second value of the lane before
      }
    }
#pragma unroll
    for (int j = 0; j < kAnyRows; ++j) {
      if (!live[j]) continue;  // the same for the whole warp
      if (odd[j]) {
#pragma unroll
        for (int i = 0; i < kAnyPairs; ++i) {
          const uint32_t right = __shfl_down_sync(0xffffffffu, x[j][i], 1);
          const uint32_t first = __shfl_sync(0xffffffffu, x[j][i + 1], 0);
          x[j][i] = __funnelshift_r(x[j][i], lane < 31 ? right : first, 16);
        }
      }
#pragma unroll
      for (int i = 0; i < kAnyPairs; ++i) {
        lo[i] = fmaf(w[j], __uint_as_float(x[j][i] << 16), lo[i]);
        hi[i] = fmaf(w[j], __uint_as_float(x[j][i] & 0xFFFF0000u), hi[i]);
      }
    }
  }
  uint16_t* o = out + m * ldo + n0;
  const bool shifted = (reinterpret_cast<uintptr_t>(o) & 2) != 0;
  uint32_t v[kAnyPairs];
#pragma unroll
  for (int i = 0; i < kAnyPairs; ++i) v[i] = pack_bf16(lo[i], hi[i]);
#pragma unroll
  for (int i = 0; i < kAnyPairs; ++i) {
    const int c = 64 * i + 2 * lane;
    if (!shifted) {
      if (c + 1 < cols)
        reinterpret_cast<uint32_t*>(o)[32 * i + lane] = v[i];
      else if (c < cols)
        o[c] = static_cast<uint16_t>(v[i]);
    } else {
      // The word of columns c - 1 and c: the pair before's second value and this one's first.
      const uint32_t left = __shfl_up_sync(0xffffffffu, v[i], 1);
      const uint32_t last = i > 0 ? __shfl_sync(0xffffffffu, v[i > 0 ? i - 1 : 0], 31) : 0u;
      const uint32_t word = __funnelshift_r(lane > 0 ? left : last, v[i], 16);
      if (c == 0)
        o[0] = static_cast<uint16_t>(v[0]);
      else if (c < cols)
        *reinterpret_cast<uint32_t*>(o + c - 1) = word;
      if (c + 2 == cols) o[c + 1] = static_cast<uint16_t>(v[i] >> 16);
    }
  }
}

// One chunk (one launch) up to 4096 choices (7.1 us there either way), else chunks of
// 1024 while there are at most 128 of them: 131072 choices of 256 experts in 10.7 us,
// in chunks of 4096 some 4 us more.
constexpr int kSortMinChunk = 4096;
constexpr int kSortMaxChunks = 128;

int64_t sort_chunk(int64_t n) {
  if (n <= kSortMinChunk) return n < 1 ? 1 : n;
  return std::max<int64_t>(kSortThreads, ((n + kSortMaxChunks - 1) / kSortMaxChunks + 1023) / 1024 * 1024);
}

int64_t expert_sort_chunks(int64_t n) { return n < 1 ? 1 : (n + sort_chunk(n) - 1) / sort_chunk(n); }

template <bool kWide>
cudaError_t sort_typed(const void* ids, int64_t n, int k, int E, int32_t* offsets, int32_t* rows, int32_t* pos,
                       int32_t* counts, cudaStream_t stream) {
  static thread_local int configured_for = -1;
  int dev = 0;
  cudaError_t st = cudaGetDevice(&dev);
  if (st != cudaSuccess) return st;
  if (configured_for != dev) {
    const int most = kSortWarps * kMx4MaxExperts * 4;
    for (auto f : {expert_sort_kernel<kWide, kSingle>, expert_sort_kernel<kWide, kCount>,
                   expert_sort_kernel<kWide, kPlace>}) {
      st = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
      if (st != cudaSuccess) return st;
    }
    configured_for = dev;
  }
  const int chunk = static_cast<int>(sort_chunk(n));
  const unsigned int grid = static_cast<unsigned int>(expert_sort_chunks(n));
  const size_t smem = static_cast<size_t>(kSortWarps) * E * 4;
  const int ni = static_cast<int>(n);
  int bits = 1;
  while ((E >> bits) != 0) ++bits;  // ids 0 .. E, E for the ones left out
  if (grid == 1)
    return launch_pdl(expert_sort_kernel<kWide, kSingle>, 1u, kSortThreads, smem, stream, ids, ni, k, E, bits, chunk,
                      offsets, rows, pos, counts);
  st = launch_pdl(expert_sort_kernel<kWide, kCount>, grid, kSortThreads, smem, stream, ids, ni, k, E, bits, chunk, offsets,
                  rows, pos, counts);
  if (st != cudaSuccess) return st;
  return launch_pdl(expert_sort_kernel<kWide, kPlace>, grid, kSortThreads, smem, stream, ids, ni, k, E, bits, chunk, offsets,
                    rows, pos, counts);
}

}  // namespace

int64_t expert_sort_counts(int64_t n, int64_t E) { return (expert_sort_chunks(n) + 3) / 4 * 4 * E; }

cudaError_t launch_expert_sort(const void* ids, bool wide, int64_t n, int k, int E, int32_t* offsets, int32_t* rows,
                               int32_t* pos, int32_t* counts, cudaStream_t stream) {
  return wide ? sort_typed<true>(ids, n, k, E, offsets, rows, pos, counts, stream)
              : sort_typed<false>(ids, n, k, E, offsets, rows, pos, counts, stream);
}

cudaError_t launch_expert_combine(const uint16_t* Y, int64_t T, int64_t N, int64_t ldy, const int32_t* pos,
                                  const float* weights, int64_t M, int k, uint16_t* out, int64_t ldo,
                                  cudaStream_t stream) {
  if (M == 0) return cudaSuccess;
  if (N % 8 == 0 && ldy % 8 == 0 && ldo % 8 == 0) {
    const int64_t grid = (M * (N / 8) + kCombineThreads - 1) / kCombineThreads;
    return launch_pdl(expert_combine_kernel, static_cast<unsigned int>(grid), kCombineThreads, 0, stream, Y, T, N, ldy,
                      pos, weights, M, k, out, ldo);
  }
  constexpr int kWindow = 64 * kAnyPairs;
  const int64_t grid = (M * ((N + kWindow - 1) / kWindow) + 3) / 4;
  return launch_pdl(expert_combine_any_kernel, static_cast<unsigned int>(grid), kCombineThreads, 0, stream, Y, T, N,
                    ldy, pos, weights, M, k, out, ldo);
}

}  // namespace spense
