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
// its run 32 choices at a time and finds the equal ones among them with one
// match instruction, so nothing depends on the order in which warps or CTAs
// arrive and the result is the stable one.
//   kSingle  the one chunk: counts, offsets and positions in one launch.
//   kCount   counts of a chunk into counts[chunk][E].
//   kPlace   recounts the chunk, takes its bases from all chunks' counts.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
enum SortMode { kSingle, kCount, kPlace };

template <bool kWide>
__device__ __forceinline__ int expert_of(const void* ids, int i, int end, int E) {
  if (i >= end) return E;
  if constexpr (kWide) {
    const long long v = __ldg(static_cast<const long long*>(ids) + i);
    return v >= 0 && v < E ? static_cast<int>(v) : E;
  } else {
    const int v = __ldg(static_cast<const int*>(ids) + i);
    return v >= 0 && v < E ? v : E;
  }
}

template <bool kWide, SortMode kMode>
__global__ void __launch_bounds__(kSortThreads)
    expert_sort_kernel(const void* __restrict__ ids, int n, int k, int E, int chunk, int32_t* __restrict__ offsets,
                       int32_t* __restrict__ rows, int32_t* __restrict__ pos, int32_t* __restrict__ counts) {
  extern __shared__ int hist[];  // [warps][E]: the warp's choices of an expert, then its first position
  __shared__ int warp_sum[kSortWarps];
  __shared__ int total_live;
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
  for (int b = i0; b < i1; b += 32) {
    const int e = expert_of<kWide>(ids, b + lane, i1, E);
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e < E && (same & below) == 0u) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // Thread t: the expert t (E <= 1024). Its choices in this chunk, and before it.
  const int t = threadIdx.x;
  int sum = 0, before = 0;
  if (t < E) {
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = hist[w * E + t];
      hist[w * E + t] = sum;
      sum += c;
    }
  }
  if constexpr (kMode == kCount) {
    if (t < E) counts[blockIdx.x * E + t] = sum;
    return;
  }
  int total = sum;
  if constexpr (kMode == kPlace) {
    total = 0;
    if (t < E)
      for (int c = 0; c < static_cast<int>(gridDim.x); ++c) {
        const int v = __ldcg(counts + c * E + t);
        if (c < static_cast<int>(blockIdx.x)) before += v;
        total += v;
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
    for (int w = 0; w < kSortWarps; ++w) hist[w * E + t] += first + before;
  }
  if (blockIdx.x == 0 && t == 0) offsets[E] = total_live;
  __syncthreads();
  for (int b = i0; b < i1; b += 32) {
    const int i = b + lane;
    const int e = expert_of<kWide>(ids, i, i1, E);
    const uint32_t same = __match_any_sync(0xffffffffu, e);
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
  }
  // The slots behind the last expert's (as many as there are choices left out).
  for (int i = total_live + blockIdx.x * kSortThreads + t; i < n; i += gridDim.x * kSortThreads) rows[i] = -1;
}

// ---------------------------------------------------------------- combine
// out[m][n] = bf16(sum over j of weights[m][j] * Y[pos[m][j]][n]) in fp32, j
// ascending, choices with pos outside [0, T) left out (their weight is not
// looked at). Bound by the gathered rows' bytes.
constexpr int kCombineThreads = 128;

__device__ __forceinline__ void fma8(float (&acc)[8], const uint4& v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, __uint_as_float(u[i] << 16), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, __uint_as_float(u[i] & 0xFFFF0000u), acc[2 * i + 1]);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// kVec: eight columns a thread (rows 16-byte aligned); else one.
template <bool kVec>
__global__ void __launch_bounds__(kCombineThreads)
    expert_combine_kernel(const uint16_t* __restrict__ Y, int64_t T, int64_t N, int64_t ldy,
                          const int32_t* __restrict__ pos, const float* __restrict__ weights, int k,
                          uint16_t* __restrict__ out, int64_t ldo) {
  constexpr int kCols = kVec ? 8 : 1;
  pdl_trigger();
  const int64_t spans = (N + kCombineThreads * kCols - 1) / (kCombineThreads * kCols);
  const int64_t m = blockIdx.x / spans;
  const int64_t n = (blockIdx.x - m * spans) * (kCombineThreads * kCols) + threadIdx.x * kCols;
  pdl_wait();
  if (n >= N) return;
  float acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
  const int32_t* pm = pos + m * k;
  const float* wm = weights + m * k;
  for (int j0 = 0; j0 < k; j0 += 8) {
    float w[8];
    bool live[8];
    uint4 v[kVec ? 8 : 1];
    uint16_t s[kVec ? 1 : 8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      live[j] = false;
      if (j0 + j < k) {
        const int64_t p = __ldg(pm + j0 + j);
        live[j] = p >= 0 && p < T;
        if (live[j]) {
          w[j] = __ldg(wm + j0 + j);
          if constexpr (kVec)
            v[j] = __ldg(reinterpret_cast<const uint4*>(Y + p * ldy + n));
          else
            s[j] = __ldg(Y + p * ldy + n);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (live[j]) {
        if constexpr (kVec)
          fma8(acc, v[j], w[j]);
        else
          acc[0] = fmaf(w[j], __uint_as_float(static_cast<uint32_t>(s[j]) << 16), acc[0]);
      }
  }
  if constexpr (kVec) {
    *reinterpret_cast<uint4*>(out + m * ldo + n) = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                                                              pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
  } else {
    out[m * ldo + n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[0]));
  }
}

constexpr int kSortMinChunk = 4096;  // one chunk (one launch) up to here
constexpr int kSortMaxChunks = 128;

int64_t sort_chunk(int64_t n) {
  if (n <= kSortMinChunk) return n < 1 ? 1 : n;
  return std::max<int64_t>(kSortThreads, ((n + kSortMaxChunks - 1) / kSortMaxChunks + 1023) / 1024 * 1024);
}

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
  if (grid == 1)
    return launch_pdl(expert_sort_kernel<kWide, kSingle>, 1u, kSortThreads, smem, stream, ids, ni, k, E, chunk,
                      offsets, rows, pos, counts);
  st = launch_pdl(expert_sort_kernel<kWide, kCount>, grid, kSortThreads, smem, stream, ids, ni, k, E, chunk, offsets,
                  rows, pos, counts);
  if (st != cudaSuccess) return st;
  return launch_pdl(expert_sort_kernel<kWide, kPlace>, grid, kSortThreads, smem, stream, ids, ni, k, E, chunk, offsets,
                    rows, pos, counts);
}

}  // namespace

int64_t expert_sort_chunks(int64_t n) { return n < 1 ? 1 : (n + sort_chunk(n) - 1) / sort_chunk(n); }

cudaError_t launch_expert_sort(const void* ids, bool wide, int64_t n, int k, int E, int32_t* offsets, int32_t* rows,
                               int32_t* pos, int32_t* counts, cudaStream_t stream) {
  return wide ? sort_typed<true>(ids, n, k, E, offsets, rows, pos, counts, stream)
              : sort_typed<false>(ids, n, k, E, offsets, rows, pos, counts, stream);
}

cudaError_t launch_expert_combine(const uint16_t* Y, int64_t T, int64_t N, int64_t ldy, const int32_t* pos,
                                  const float* weights, int64_t M, int k, uint16_t* out, int64_t ldo,
                                  cudaStream_t stream) {
  if (M == 0) return cudaSuccess;
  const bool vec = N % 8 == 0 && ldy % 8 == 0 && ldo % 8 == 0;
  const int64_t per = kCombineThreads * (vec ? 8 : 1);
  const unsigned int grid = static_cast<unsigned int>(M * ((N + per - 1) / per));
  return vec ? launch_pdl(expert_combine_kernel<true>, grid, kCombineThreads, 0, stream, Y, T, N, ldy, pos, weights, k,
                          out, ldo)
             : launch_pdl(expert_combine_kernel<false>, grid, kCombineThreads, 0, stream, Y, T, N, ldy, pos, weights,
                          k, out, ldo);
}

}  // namespace spense
