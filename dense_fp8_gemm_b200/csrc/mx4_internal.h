// Internal declarations of the MXFP4 and expert operators. Not part of the
// public ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace spense {

// A packed MXFP4 weight block: 128 rows x 256 columns. Codes first, 128 bytes a
// row in the 128-byte swizzle, then the scales of the block's two column groups
// of 128: 32 lanes x 4 words, word w of lane l the four scale bytes of row
// 32 w + l (the order tcgen05.cp moves into tensor memory).
constexpr int kMx4Rows = 128;
constexpr int kMx4Cols = 256;
constexpr int kMx4CodeBytes = 16384;
constexpr int kMx4ScaleBytes = 1024;
constexpr int kMx4BlockBytes = kMx4CodeBytes + kMx4ScaleBytes;

constexpr int kMx4BarrierBytes = 512;  // mbarriers and flags behind the ring
constexpr int kMx4XsSlots = 8;  // blocks whose activation scales are ahead of the products
constexpr int kMx4XsTileBytes = 2048;  // scales of a block for up to 256 rows, in tcgen05.cp's order
constexpr int kMx4MaxExperts = 1024;
constexpr int64_t kMx4MaxRows = 1 << 20;

struct Mx4GemmParams {
  const uint8_t* blocks;
  const uint32_t* xs;      // activation scale words [groups][T]
  uint16_t* y;
  int64_t ldy;
  const int32_t* offsets;  // device int32 [E + 1], or NULL: one expert with all T rows
  unsigned int* status;
  const unsigned int* test_gate;  // test build only: loaders wait (bounded) until this word is nonzero
  int E, N, T;
  int n_tiles, kblocks, groups;
  int last_steps;          // K = 64 steps in the last block (1 .. 4)
  int npad;                // rows of activations per tile (MMA N), a multiple of 16
  int box[3];              // rows one activation load covers, smallest first; box[2]: a CTA's share of npad
  int group;               // row tiles that all weight tiles pass before the next ones
  int stages, nacc;
  int bps;                 // blocks a stage holds (1 or 2)
  int pair;                // 1: CTA pairs (tcgen05 cta_group::2) share 256-row MMAs
  int split;               // CTAs of a cluster sharing one tile's K range (1: none)
  uint32_t stage_bytes, xs_bytes, tmem_cols;  // bytes of a stage, of a slot of activation scales
  int w_keep;              // 1: weights are read again by later tiles, keep them in L2
};

// Tensor maps of a launch: the activation codes in three box heights, and the
// scale words as one array in boxes of 64 and 256 words.
struct Mx4GemmMaps {
  CUtensorMap x[3];
  CUtensorMap xs_narrow, xs_wide;
  CUtensorMap w, xs_tiles;  // pair mode: the packed blocks and the scale tiles, as rows of 128 bytes
};

constexpr int kMx4MaxTile = 240;  // rows a tile takes: with three words in front, one box of 256 scale words
constexpr int kMx4PairRows = 256;  // the same of a pair, the most an MMA takes

struct Mx4GemmPlan {
  int npad, stages, nacc, bps, pair, split, grid;
  int64_t row_tiles;  // row tiles at most (all experts)
  size_t workspace_bytes;
  uint32_t stage_bytes, xs_bytes, tmem_cols, smem_bytes;
};

cudaError_t launch_mx4_gemm(const Mx4GemmMaps& maps, const Mx4GemmParams& p, int grid, uint32_t smem_bytes,
                            cudaStream_t stream);

// Clusters of `cluster` CTAs with that much shared memory the device holds at once.
cudaError_t mx4_max_clusters(int cluster, uint32_t smem_bytes, int* out);
// Pair mode: the activation scales of p's row tiles in tcgen05.cp's order.
cudaError_t launch_mx4_scale_tiles(const Mx4GemmParams& p, int row_tiles, uint32_t* out, cudaStream_t stream);

// x_type: SPENSE_TYPE_*. rows: gather index [T] or NULL. words: scales as words.
cudaError_t launch_mx4_quantize(const void* X, int x_type, int64_t T, int64_t K, int64_t ldx, const int32_t* rows,
                                int64_t M_src, uint8_t* Xq, uint8_t* xs, bool words, int sms, cudaStream_t stream);
cudaError_t launch_mx4_dequantize(const uint8_t* Xq, const uint8_t* xs, bool words, int64_t T, int64_t K, void* Y,
                                  int y_type, int sms, cudaStream_t stream);
cudaError_t launch_mx4_pack(const uint8_t* Wq, const uint8_t* ws, int64_t E, int64_t N, int64_t K, int n_tiles,
                            int kblocks, uint8_t* blocks, unsigned int* err, cudaStream_t stream);

// int32 counters expert_sort keeps in its workspace.
int64_t expert_sort_counts(int64_t n, int64_t E);
cudaError_t launch_expert_sort(const void* ids, bool wide, int64_t n, int k, int E, int32_t* offsets, int32_t* rows,
                               int32_t* pos, int32_t* counts, cudaStream_t stream);
cudaError_t launch_expert_combine(const uint16_t* Y, int64_t T, int64_t N, int64_t ldy, const int32_t* pos,
                                  const float* weights, int64_t M, int k, uint16_t* out, int64_t ldo,
                                  cudaStream_t stream);

}  // namespace spense
