// MXFP4 quantisation, dequantisation and weight packing.
//
// The OCP Microscaling (MX) format with 4-bit elements: 32 consecutive columns
// of a row share a power-of-two scale 2^e (one byte, e + 127; 255 is NaN) and
// each value is a sign and one of 0, 1/2, 1, 3/2, 2, 3, 4, 6 (e2m1). The
// quantiser takes e = floor(log2 max|x|) - 2 of the block, so the largest value
// lands in [4, 8) and only the part above 6 saturates; x 2^-e is exact (a power
// of two, and what underflows rounds to code 0 either way), so the one rounding
// is to the nearest code, ties to even.
//
// All three kernels are copies with a little arithmetic: bound by HBM for many
// rows, by launch and load latency for few.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mx4_internal.h"
#include "pdl.cuh"
#include "spense.h"

namespace spense {
namespace {

constexpr int kThreads = 256;

// kN 16-byte pieces of consecutive values as floats (exact for every input type).
template <int kType, int kN>
__device__ __forceinline__ void to_floats(const uint4 (&raw)[kN], float* f) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kType == SPENSE_TYPE_F32) {
        f[4 * i + j] = __uint_as_float(w[j]);
      } else if constexpr (kType == SPENSE_TYPE_BF16) {
        f[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        f[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      } else {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        f[8 * i + 2 * j] = v.x;
        f[8 * i + 2 * j + 1] = v.y;
      }
    }
  }
}

// Eight floats -> eight e2m1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* f) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// The work of both kernels. A thread takes 16 columns, two threads a block, eight a scale word
// (128 columns), a warp 512 columns.
//   kWide (many rows): the eight warps of a CTA take eight rows and each two such
//     pieces of its row, all loads first. The CTA's scale words leave through
//     shared memory, eight rows' words of a column group (32 bytes) at a time:
//     written one by one they were twice as many requests as the codes. 32768
//     gathered rows of 5120 take 55 us (the rows' four readings from L2 bound it; with
//     eight columns a thread and single words 90 us), 8192 rows in order 17.4 us (f16
//     the same, f32 29 us, which is HBM's rate; gathered f16 56 us, f32 94).
//   else (few rows): the eight warps take eight pieces of one row, so a token's
//     5120 columns are two CTAs with one round of loads.
template <bool kWide>
struct RowTile {
  static constexpr int kPieces = kWide ? 2 : 1;
  static constexpr int kRows = kWide ? 8 : 1;
  static constexpr int kCols = kWide ? 1024 : 4096;
  static unsigned int grid(int64_t T, int64_t K) {
    return static_cast<unsigned int>(((T + kRows - 1) / kRows) * ((K + kCols - 1) / kCols));
  }
};

template <int kType, bool kWide>
__global__ void __launch_bounds__(kThreads)
    mx4_quantize_kernel(const void* X, int T, int K, int64_t ldx, const int32_t* rows,
                        int M_src, uint8_t* __restrict__ Xq, uint8_t* __restrict__ xs, int words) {
  using Q = RowTile<kWide>;
  constexpr int kSize = kType == SPENSE_TYPE_F32 ? 4 : 2;
  constexpr int kLoads = kSize;  // 16-byte loads for 16 values
  __shared__ uint32_t staged[kWide ? 64 : 1];  // [column group][row]
  __shared__ int live_row[kWide ? 8 : 1];
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned int spans = static_cast<unsigned int>((K + Q::kCols - 1) / Q::kCols);
  const unsigned int rb = blockIdx.x / spans;
  const int span0 = static_cast<int>(blockIdx.x - rb * spans) * Q::kCols;
  const int row0 = static_cast<int>(rb) * Q::kRows;
  const int row = row0 + (kWide ? warp : 0);
  const int col0 = span0 + (kWide ? 0 : warp * 512) + lane * 16;
  pdl_wait();
  int src = -1;  // the warp's source row, or none
  if (row < T) {
    src = rows != nullptr ? ld_dep(rows + row) : row;
    if (src >= M_src) src = -1;
  }
  const char* xrow = static_cast<const char*>(X) + static_cast<int64_t>(src) * ldx * kSize;
  uint4 raw[Q::kPieces][kLoads];
#pragma unroll
  for (int i = 0; i < Q::kPieces; ++i) {
    const int c = col0 + 512 * i;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      raw[i][j] = make_uint4(0u, 0u, 0u, 0u);
      if (src >= 0 && c < K) raw[i][j] = ld_dep(reinterpret_cast<const uint4*>(xrow + c * kSize) + j);
    }
  }
#pragma unroll
  for (int i = 0; i < Q::kPieces; ++i) {
    const int c = col0 + 512 * i;
    // The largest magnitude of the thread's 16 values as a float's bit pattern:
    // patterns are ordered like the values, infinities and NaN above all. 16-bit
    // types compare their own patterns, two at a time.
    uint32_t m;
    if constexpr (kType == SPENSE_TYPE_F32) {
      m = 0u;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        m = max(max(m, max(raw[i][j].x & 0x7FFFFFFFu, raw[i][j].y & 0x7FFFFFFFu)),
                max(raw[i][j].z & 0x7FFFFFFFu, raw[i][j].w & 0x7FFFFFFFu));
    } else {
      uint32_t p = 0u;
#pragma unroll
      for (int j = 0; j < kLoads; ++j)
        p = __vmaxu2(__vmaxu2(p, __vmaxu2(raw[i][j].x & 0x7FFF7FFFu, raw[i][j].y & 0x7FFF7FFFu)),
                     __vmaxu2(raw[i][j].z & 0x7FFF7FFFu, raw[i][j].w & 0x7FFF7FFFu));
      p = max(p & 0xFFFFu, p >> 16);
      m = kType == SPENSE_TYPE_BF16 ? p << 16
                                    : __float_as_uint(__half2float(__ushort_as_half(static_cast<uint16_t>(p))));
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    // Scale byte e + 127 = (biased exponent of the largest magnitude) - 2, from
    // below cut at 0 (zeros, subnormals); 255 marks a block that is not finite.
    const uint32_t ex = m >> 23;
    const uint32_t byte = ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
    const uint32_t inv = byte == 255u ? 0x3F800000u : (254u - byte) << 23;  // 2^-e as a float
    float f[16];
    if constexpr (kType == SPENSE_TYPE_BF16) {
      // 2^-e and x 2^-e are bf16 values (its exponents are fp32's): two products at once.
      const uint32_t two = inv | (inv >> 16);
      const __nv_bfloat162 inv2 = *reinterpret_cast<const __nv_bfloat162*>(&two);
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const uint32_t w[4] = {raw[i][j].x, raw[i][j].y, raw[i][j].z, raw[i][j].w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[h]), inv2);
          const uint32_t u = *reinterpret_cast<const uint32_t*>(&v);
          f[8 * j + 2 * h] = __uint_as_float(u << 16);
          f[8 * j + 2 * h + 1] = __uint_as_float(u & 0xFFFF0000u);
        }
      }
    } else {
      to_floats<kType, kLoads>(raw[i], f);
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] *= __uint_as_float(inv);
    }
    const bool live = src >= 0 && c < K;
    if (live)
      *reinterpret_cast<uint2*>(Xq + (static_cast<int64_t>(row) * K + c) / 2) =
          make_uint2(cvt_e2m1x8(f), cvt_e2m1x8(f + 8));
    if (words) {
      uint32_t v = c < K ? byte << (8 * ((lane >> 1) & 3)) : 0u;  // bytes past K are 0
      v |= __shfl_xor_sync(0xffffffffu, v, 2);
      v |= __shfl_xor_sync(0xffffffffu, v, 4);
      if constexpr (kWide) {
        if ((lane & 7) == 0) staged[(4 * i + (lane >> 3)) * 8 + warp] = v;
      } else {
        if ((lane & 7) == 0 && live) reinterpret_cast<uint32_t*>(xs)[static_cast<int64_t>(c / 128) * T + row] = v;
      }
    } else if ((lane & 1) == 0 && live) {
      xs[static_cast<int64_t>(row) * (K / 32) + c / 32] = static_cast<uint8_t>(byte);
    }
  }
  if constexpr (kWide) {
    if (words) {  // the same for the whole grid
      if (lane == 0) live_row[warp] = src >= 0;
      __syncthreads();
      const int t = threadIdx.x, g = span0 / 128 + (t >> 3), r = t & 7;
      if (t < 64 && g * 128 < K && live_row[r])
        reinterpret_cast<uint32_t*>(xs)[static_cast<int64_t>(g) * T + row0 + r] = staged[t];
    }
  }
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : (byte == 0u ? 0x00400000u : byte << 23));
}

// Eight codes -> eight values of magnitude 0 .. 6 as floats.
__device__ __forceinline__ void e2m1x8_to_float(uint32_t codes, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h2;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
        : "=r"(h2)
        : "r"(codes >> (8 * i)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

// 32-byte store (address 32-byte aligned).
__device__ __forceinline__ void st_global_v8(void* ptr, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(ptr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Dequantiser. A thread takes 16 columns (half a block: one scale, 32 bytes of bf16
// output in one store when the output is 32-byte aligned), a warp 512 columns of a
// row; kWide: eight rows a CTA, two pieces a warp, all loads first; else eight
// pieces of one row. 32768 rows of 5120 take 71 us, 6.0 TB/s (16-byte stores 86 us);
// as fp32, whose 64 bytes a thread leave in 16-byte stores, 178 us, 4.3 TB/s.
//
// Every value is exact in the output type (two significant bits; 2^-128 at least)
// below 2^128; larger ones (4 and 6 times 2^126, 2 and more times 2^127), which the
// quantiser never makes, become infinite.
template <bool kF32, bool kWide>
__global__ void __launch_bounds__(kThreads)
    mx4_dequantize_kernel(const uint8_t* Xq, const uint8_t* xs, int words, int T, int K,
                          void* __restrict__ Y) {
  using Q = RowTile<kWide>;
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned int spans = static_cast<unsigned int>((K + Q::kCols - 1) / Q::kCols);
  const unsigned int rb = blockIdx.x / spans;
  const int row = static_cast<int>(rb) * Q::kRows + (kWide ? warp : 0);
  const int col0 = static_cast<int>(blockIdx.x - rb * spans) * Q::kCols + (kWide ? 0 : warp * 512) + lane * 16;
  pdl_wait();
  if (row >= T) return;
  uint2 codes[Q::kPieces];
  uint32_t byte[Q::kPieces];
#pragma unroll
  for (int i = 0; i < Q::kPieces; ++i) {
    const int c = col0 + 512 * i;
    codes[i] = make_uint2(0u, 0u);
    byte[i] = 0u;
    if (c < K) {
      codes[i] = ld_dep(reinterpret_cast<const uint2*>(Xq + (static_cast<int64_t>(row) * K + c) / 2));
      byte[i] = words ? ld_dep(xs + (static_cast<int64_t>(c / 128) * T + row) * 4 + (c / 32) % 4)
                      : ld_dep(xs + static_cast<int64_t>(row) * (K / 32) + c / 32);
    }
  }
#pragma unroll
  for (int i = 0; i < Q::kPieces; ++i) {
    const int c = col0 + 512 * i;
    if (c >= K) break;
    const float s = scale_value(byte[i]);
    const int64_t at = static_cast<int64_t>(row) * K + c;
    uint32_t o[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[8];
      e2m1x8_to_float(h == 0 ? codes[i].x : codes[i].y, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] *= s;
      if constexpr (kF32) {
        float4* y = reinterpret_cast<float4*>(static_cast<float*>(Y) + at + 8 * h);
        y[0] = make_float4(f[0], f[1], f[2], f[3]);
        y[1] = make_float4(f[4], f[5], f[6], f[7]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
          o[4 * h + j] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
    }
    if constexpr (!kF32) {
      uint16_t* y = static_cast<uint16_t*>(Y) + at;
      if ((reinterpret_cast<uintptr_t>(Y) & 31) == 0) {
        st_global_v8(y, o);
      } else {
        reinterpret_cast<uint4*>(y)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4*>(y)[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

// One CTA a block of the packed layout (see mx4_internal.h). Rows past N and
// columns past K hold code 0 with scale byte 0. Runs once per weight.
__global__ void __launch_bounds__(kThreads)
    mx4_pack_kernel(const uint8_t* __restrict__ Wq, const uint8_t* __restrict__ ws, int64_t N, int64_t K, int n_tiles,
                    int kblocks, uint8_t* __restrict__ blocks, unsigned int* err) {
  const int64_t b = blockIdx.x;
  const int kb = static_cast<int>(b % kblocks);
  const int64_t et = b / kblocks;
  const int nt = static_cast<int>(et % n_tiles);
  const int64_t e = et / n_tiles;
  uint8_t* out = blocks + b * kMx4BlockBytes;
  for (int i = threadIdx.x; i < kMx4CodeBytes / 16; i += kThreads) {
    const int r = i >> 3, c = i & 7;
    const int64_t n = static_cast<int64_t>(nt) * kMx4Rows + r, byte = static_cast<int64_t>(kb) * 128 + c * 16;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (n < N && byte < K / 2) v = __ldg(reinterpret_cast<const uint4*>(Wq + (e * N + n) * (K / 2) + byte));
    *reinterpret_cast<uint4*>(out + r * 128 + ((c ^ (r & 7)) << 4)) = v;
  }
  {
    const int r = threadIdx.x & 127, j = threadIdx.x >> 7;
    const int64_t n = static_cast<int64_t>(nt) * kMx4Rows + r;
    uint32_t v = 0;
    for (int q = 0; q < 4; ++q) {
      const int64_t blk = static_cast<int64_t>(kb) * 8 + j * 4 + q;
      if (n < N && blk < K / 32) {
        const uint32_t s = __ldg(ws + (e * N + n) * (K / 32) + blk);
        if (s == 255u) atomicOr(err, 1u);
        v |= s << (8 * q);
      }
    }
    *reinterpret_cast<uint32_t*>(out + kMx4CodeBytes + j * 512 + (r & 31) * 16 + (r >> 5) * 4) = v;
  }
}

template <int kType>
cudaError_t quantize_typed(const void* X, int64_t T, int64_t K, int64_t ldx, const int32_t* rows, int64_t M_src,
                           uint8_t* Xq, uint8_t* xs, bool words, int sms, cudaStream_t stream) {
  const int t = static_cast<int>(T), k = static_cast<int>(K), m = static_cast<int>(M_src), w = words ? 1 : 0;
  // Eight rows a CTA once that fills the device twice over.
  if (RowTile<true>::grid(T, K) >= 2u * static_cast<unsigned int>(sms))
    return launch_pdl(mx4_quantize_kernel<kType, true>, RowTile<true>::grid(T, K), kThreads, 0, stream, X, t, k, ldx,
                      rows, m, Xq, xs, w);
  return launch_pdl(mx4_quantize_kernel<kType, false>, RowTile<false>::grid(T, K), kThreads, 0, stream, X, t, k, ldx,
                    rows, m, Xq, xs, w);
}

template <bool kF32>
cudaError_t dequantize_typed(const uint8_t* Xq, const uint8_t* xs, bool words, int64_t T, int64_t K, void* Y, int sms,
                             cudaStream_t stream) {
  const int t = static_cast<int>(T), k = static_cast<int>(K), w = words ? 1 : 0;
  if (RowTile<true>::grid(T, K) >= 2u * static_cast<unsigned int>(sms))
    return launch_pdl(mx4_dequantize_kernel<kF32, true>, RowTile<true>::grid(T, K), kThreads, 0, stream, Xq, xs, w,
                      t, k, Y);
  return launch_pdl(mx4_dequantize_kernel<kF32, false>, RowTile<false>::grid(T, K), kThreads, 0, stream, Xq, xs, w,
                    t, k, Y);
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* X, int x_type, int64_t T, int64_t K, int64_t ldx, const int32_t* rows,
                                int64_t M_src, uint8_t* Xq, uint8_t* xs, bool words, int sms, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  if (x_type == SPENSE_TYPE_F32)
    return quantize_typed<SPENSE_TYPE_F32>(X, T, K, ldx, rows, M_src, Xq, xs, words, sms, stream);
  if (x_type == SPENSE_TYPE_F16)
    return quantize_typed<SPENSE_TYPE_F16>(X, T, K, ldx, rows, M_src, Xq, xs, words, sms, stream);
  return quantize_typed<SPENSE_TYPE_BF16>(X, T, K, ldx, rows, M_src, Xq, xs, words, sms, stream);
}

cudaError_t launch_mx4_dequantize(const uint8_t* Xq, const uint8_t* xs, bool words, int64_t T, int64_t K, void* Y,
                                  int y_type, int sms, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  return y_type == SPENSE_TYPE_F32 ? dequantize_typed<true>(Xq, xs, words, T, K, Y, sms, stream)
                                   : dequantize_typed<false>(Xq, xs, words, T, K, Y, sms, stream);
}

cudaError_t launch_mx4_pack(const uint8_t* Wq, const uint8_t* ws, int64_t E, int64_t N, int64_t K, int n_tiles,
                            int kblocks, uint8_t* blocks, unsigned int* err, cudaStream_t stream) {
  mx4_pack_kernel<<<static_cast<unsigned int>(E * n_tiles * kblocks), kThreads, 0, stream>>>(Wq, ws, N, K, n_tiles,
                                                                                             kblocks, blocks, err);
  return cudaGetLastError();
}

}  // namespace spense
