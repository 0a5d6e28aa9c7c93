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

// Eight consecutive values as floats (exact for every input type).
struct Raw8 {
  uint4 a, b;
};

template <int kType>
__device__ __forceinline__ Raw8 load8(const void* row, int64_t col) {
  Raw8 r;
  if constexpr (kType == SPENSE_TYPE_F32) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(row) + col);
    r.a = __ldg(s);
    r.b = __ldg(s + 1);
  } else {
    r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + col));
    r.b = make_uint4(0u, 0u, 0u, 0u);
  }
  return r;
}

template <int kType>
__device__ __forceinline__ void to_float8(const Raw8& r, float (&f)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kType == SPENSE_TYPE_F32) {
      f[2 * i] = __uint_as_float(w[2 * i]);
      f[2 * i + 1] = __uint_as_float(w[2 * i + 1]);
    } else if constexpr (kType == SPENSE_TYPE_BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    } else {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
}

// Eight floats -> eight e2m1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&f)[8]) {
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

// The work of both kernels: a warp covers 256 columns of a row at a time, eight
// a lane, so a block of 32 columns is four lanes and a scale word (128 columns)
// sixteen. kWide (many rows): the eight warps of a CTA take eight rows and each
// four such pieces of its row, all loads issued first; the CTA's scale words of
// one column group are eight consecutive words (one 32-byte sector). Otherwise
// (few rows) the eight warps take eight pieces of one row, one load a lane, so
// one token of 5120 columns spreads over three CTAs.
template <bool kWide>
struct Where {
  static constexpr int kPieces = kWide ? 4 : 1;
  static constexpr int kRowsPerCta = kWide ? 8 : 1;
  static constexpr int kColsPerCta = kWide ? 1024 : 2048;
  int64_t row;
  int64_t col0;  // this lane's first column of piece 0; piece i is 256 columns on
  __device__ Where(int64_t K) {
    const int64_t spans = (K + kColsPerCta - 1) / kColsPerCta;
    const int64_t rb = blockIdx.x / spans, sb = blockIdx.x - rb * spans;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    row = rb * kRowsPerCta + (kWide ? warp : 0);
    col0 = sb * kColsPerCta + (kWide ? 0 : warp * 256) + lane * 8;
  }
};

template <bool kWide>
unsigned int where_grid(int64_t T, int64_t K) {
  using W = Where<kWide>;
  return static_cast<unsigned int>(((T + W::kRowsPerCta - 1) / W::kRowsPerCta) *
                                   ((K + W::kColsPerCta - 1) / W::kColsPerCta));
}

template <int kType, bool kWide>
__global__ void __launch_bounds__(kThreads)
    mx4_quantize_kernel(const void* __restrict__ X, int64_t T, int64_t K, int64_t ldx,
                        const int32_t* __restrict__ rows, int64_t M_src, uint8_t* __restrict__ Xq,
                        uint8_t* __restrict__ xs, int words) {
  using W = Where<kWide>;
  pdl_trigger();
  const W w(K);
  const int lane = threadIdx.x & 31;
  pdl_wait();
  if (w.row >= T) return;
  int64_t src = w.row;
  if (rows != nullptr) {
    src = __ldg(rows + w.row);
    if (src < 0 || src >= M_src) return;  // the whole warp: the row is left as it was
  }
  const int64_t esize = kType == SPENSE_TYPE_F32 ? 4 : 2;
  const void* xrow = static_cast<const uint8_t*>(X) + src * ldx * esize;
  Raw8 raw[W::kPieces];
#pragma unroll
  for (int i = 0; i < W::kPieces; ++i) {
    const int64_t c = w.col0 + 256 * i;
    raw[i].a = raw[i].b = make_uint4(0u, 0u, 0u, 0u);
    if (c < K) raw[i] = load8<kType>(xrow, c);
  }
#pragma unroll
  for (int i = 0; i < W::kPieces; ++i) {
    const int64_t c = w.col0 + 256 * i;
    float f[8];
    to_float8<kType>(raw[i], f);
    // Magnitudes as bit patterns: ordered like the values, infinities and NaN above all.
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // Scale byte e + 127 = (biased exponent of the largest magnitude) - 2, from
    // below cut at 0 (zeros, subnormals); 255 marks a block that is not finite.
    const uint32_t ex = m >> 23;
    const uint32_t byte = ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
    const float inv = __uint_as_float(byte == 255u ? 0x3F800000u : (254u - byte) << 23);  // 2^-e
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= inv;
    const uint32_t codes = cvt_e2m1x8(f);
    if (c < K) *reinterpret_cast<uint32_t*>(Xq + w.row * (K / 2) + c / 2) = codes;
    if (words) {
      uint32_t v = c < K ? byte << (8 * ((lane >> 2) & 3)) : 0u;  // bytes past K are 0
      v |= __shfl_xor_sync(0xffffffffu, v, 4);
      v |= __shfl_xor_sync(0xffffffffu, v, 8);
      if ((lane & 15) == 0 && c < K) reinterpret_cast<uint32_t*>(xs)[(c / 128) * T + w.row] = v;
    } else if ((lane & 3) == 0 && c < K) {
      xs[w.row * (K / 32) + c / 32] = static_cast<uint8_t>(byte);
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

// Every value is exact in the output type (three significant bits; 2^-128 at
// least) up to 6 x 2^125; larger ones, which the quantiser never makes, may
// round to infinity.
template <bool kF32, bool kWide>
__global__ void __launch_bounds__(kThreads)
    mx4_dequantize_kernel(const uint8_t* __restrict__ Xq, const uint8_t* __restrict__ xs, int words, int64_t T,
                          int64_t K, void* __restrict__ Y) {
  using W = Where<kWide>;
  pdl_trigger();
  const W w(K);
  pdl_wait();
  if (w.row >= T) return;
  uint32_t codes[W::kPieces], byte[W::kPieces];
#pragma unroll
  for (int i = 0; i < W::kPieces; ++i) {
    const int64_t c = w.col0 + 256 * i;
    codes[i] = byte[i] = 0u;
    if (c < K) {
      codes[i] = __ldg(reinterpret_cast<const uint32_t*>(Xq + w.row * (K / 2) + c / 2));
      byte[i] = words ? __ldg(xs + ((c / 128) * T + w.row) * 4 + (c / 32) % 4) : __ldg(xs + w.row * (K / 32) + c / 32);
    }
  }
#pragma unroll
  for (int i = 0; i < W::kPieces; ++i) {
    const int64_t c = w.col0 + 256 * i;
    if (c >= K) break;
    float f[8];
    e2m1x8_to_float(codes[i], f);
    const float s = scale_value(byte[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= s;
    if constexpr (kF32) {
      float4* y = reinterpret_cast<float4*>(static_cast<float*>(Y) + w.row * K + c);
      y[0] = make_float4(f[0], f[1], f[2], f[3]);
      y[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(Y) + w.row * K + c) = make_uint4(o[0], o[1], o[2], o[3]);
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
                           uint8_t* Xq, uint8_t* xs, bool words, bool wide, cudaStream_t stream) {
  return wide ? launch_pdl(mx4_quantize_kernel<kType, true>, where_grid<true>(T, K), kThreads, 0, stream, X, T, K, ldx,
                           rows, M_src, Xq, xs, static_cast<int>(words))
              : launch_pdl(mx4_quantize_kernel<kType, false>, where_grid<false>(T, K), kThreads, 0, stream, X, T, K,
                           ldx, rows, M_src, Xq, xs, static_cast<int>(words));
}

// Eight rows a CTA once that fills the device twice over.
bool wide_rows(int64_t T, int64_t K, int sms) { return where_grid<true>(T, K) >= 2u * static_cast<unsigned int>(sms); }

}  // namespace

cudaError_t launch_mx4_quantize(const void* X, int x_type, int64_t T, int64_t K, int64_t ldx, const int32_t* rows,
                                int64_t M_src, uint8_t* Xq, uint8_t* xs, bool words, int sms, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const bool wide = wide_rows(T, K, sms);
  if (x_type == SPENSE_TYPE_F32)
    return quantize_typed<SPENSE_TYPE_F32>(X, T, K, ldx, rows, M_src, Xq, xs, words, wide, stream);
  if (x_type == SPENSE_TYPE_F16)
    return quantize_typed<SPENSE_TYPE_F16>(X, T, K, ldx, rows, M_src, Xq, xs, words, wide, stream);
  return quantize_typed<SPENSE_TYPE_BF16>(X, T, K, ldx, rows, M_src, Xq, xs, words, wide, stream);
}

cudaError_t launch_mx4_dequantize(const uint8_t* Xq, const uint8_t* xs, bool words, int64_t T, int64_t K, void* Y,
                                  int y_type, int sms, cudaStream_t stream) {
  if (T == 0) return cudaSuccess;
  const bool wide = wide_rows(T, K, sms);
  const bool f32 = y_type == SPENSE_TYPE_F32;
  auto go = [&](auto kernel, unsigned int grid) {
    return launch_pdl(kernel, grid, kThreads, 0, stream, Xq, xs, static_cast<int>(words), T, K, Y);
  };
  if (f32)
    return wide ? go(mx4_dequantize_kernel<true, true>, where_grid<true>(T, K))
                : go(mx4_dequantize_kernel<true, false>, where_grid<false>(T, K));
  return wide ? go(mx4_dequantize_kernel<false, true>, where_grid<true>(T, K))
              : go(mx4_dequantize_kernel<false, false>, where_grid<false>(T, K));
}

cudaError_t launch_mx4_pack(const uint8_t* Wq, const uint8_t* ws, int64_t E, int64_t N, int64_t K, int n_tiles,
                            int kblocks, uint8_t* blocks, unsigned int* err, cudaStream_t stream) {
  mx4_pack_kernel<<<static_cast<unsigned int>(E * n_tiles * kblocks), kThreads, 0, stream>>>(Wq, ws, N, K, n_tiles,
                                                                                             kblocks, blocks, err);
  return cudaGetLastError();
}

}  // namespace spense
