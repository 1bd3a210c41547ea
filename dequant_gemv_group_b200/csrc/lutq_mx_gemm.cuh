// The product of two microscaled 4-bit matrices: what its launchers share.
#pragma once

#include <cuda.h>

#include <algorithm>

#include "lutq_mx.cuh"

namespace lutq {

// What a launch computes.  Rows of the weight matrix (A) are tensor-memory
// lanes, tokens (B) are columns.
enum MxMode {
  kMxPlain = 0,   // y[m, n] = sum_k x[m, k] w[n, k]
  kMxGateUp = 1,  // per expert: h = silu(x gate^T) * (x up^T), rounded to bf16
  kMxDown = 2,    // per expert: out = h down^T, fp32
};

struct MxGemmArgs {
  const uint8_t* a_scales[2];  // scale chunks of the weight matrices (of expert 0)
  const float* a_rows[2];      // nvfp4: their row scales
  int64_t a_stride;            // bytes from one expert's matrix to the next
  const uint8_t* b_scales;     // tokens: scale chunks and row scales
  const float* b_rows;
  const void* x;               // tokens quantized in the kernel: their values
  int x_dtype;
  void* y;
  int y_dtype;
  int32_t* dev_status;
  int64_t N, M, K;
  int chunks;                  // ceil(K / 256)
  int mtiles;                  // ceil(N / 128)
  int stages;
  // experts: how many tokens each has and their first rows (multiples of 128)
  const int32_t* counts;
  const int32_t* bases;
  int experts;
};

// The kernel for packed tokens (lutq_mx_gemm.cu).  tmaps: weights (two for
// gate and up), tokens in boxes of nt and of 16 rows; tiles: of the launch.
cudaError_t launch_mx_gemm(const CUtensorMap* tmaps, const MxGemmArgs& a, int fmt, int mode,
                           int nt, int64_t tiles, int num_sms, cudaStream_t stream);

// The kernel for few tokens given as values (lutq_mx_small.cu): g.x, M <= 16
// rows; or experts, with the pairs' ids.
bool mx_small_fits(int64_t pairs, int experts);
cudaError_t launch_mx_small(MxGemmArgs g, const void* weights, const void* weights2, int fmt,
                            int mode, const int32_t* ids, int pairs, int top_k, int num_sms,
                            cudaStream_t stream);

// Tensor map of `batch` matrices of packed codes, `stride` bytes apart.
cudaError_t make_mx_map(CUtensorMap* map, const void* codes, int64_t rows, int64_t K,
                        int64_t batch, int64_t stride, int box_rows);

// Their scale chunks: rows of 1024 bytes, one or two a chunk.
cudaError_t make_mx_scale_map(CUtensorMap* map, const void* packed, int64_t rows, int64_t K,
                              int64_t batch, int64_t stride, int fmt);
// An output [M, N], in boxes of 32 columns x 32 rows.
cudaError_t make_mx_out_map(CUtensorMap* map, void* y, int64_t M, int64_t N, int dtype);

// The division of a plain product among block pairs (lutq_mx_pair.cu).
struct MxPairPlan {
  int width;      // columns of the widest tile: all tokens, or the most that a tile has
  int64_t tiles;
  int split;      // pairs that share a tile by K; more than one: each tile has its own
  int tall;       // tiles of 512 weight rows instead of 256
  int pairs;      // pairs of blocks in the launch
  int slices;     // a warp's staged slices
};
MxPairPlan mx_pair_plan(int64_t M, int64_t N, int64_t K, int fmt, int num_sms);

// The kernel for many tokens (lutq_mx_pair.cu).  tiles: of experts, at most.
struct MxPairMaps {
  CUtensorMap a[2], b, b16, sa[2], sb, y;
};
cudaError_t launch_mx_pair(const MxGemmArgs& g, const void* weights, const void* weights2,
                           int64_t w_bytes, const void* tokens, int64_t token_rows, int fmt,
                           int mode, int64_t tiles, int num_sms, cudaStream_t stream);

// Tokens per tile of mx_gemm_kernel: one tile for up to 128.
int mx_tile_tokens(int64_t M);

// Clusters of s blocks (1, 2, 4, 8) that run at once, per_sm blocks on a
// multiprocessor.  Clusters of more than two leave multiprocessors over: the
// 148 hold 33 clusters of 4 and 15 of 8, or 32 of 8 at two blocks each; one
// more waits for another to end (74 tiles of 2048 x 128 split by 4 at two
// blocks each: 15.6 us, not split 7.5).  These counts are one board's, and
// others may hold one more or less; that costs time, never a tile, and a rule
// in constants gives the same sums on all boards.
inline int64_t mx_clusters(int s, int per_sm, int num_sms) {
  if (s <= 2) return int64_t(num_sms) * per_sm / s;
  return std::max(1, num_sms * (s == 4 ? 33 * per_sm : per_sm == 2 ? 32 : 15) / 148);
}

// Split a tile's K over a cluster while that gives idle multiprocessors work
// and every block a chunk.
inline int mx_split(int64_t tiles, int chunks, int per_sm, int num_sms, int most) {
  int s = 1;
  while (s < most && tiles <= mx_clusters(2 * s, per_sm, num_sms) && chunks >= 2 * s) s *= 2;
  return s;
}

// A block that holds c of an SM's 512 columns of tensor memory asks for at
// least c / 512 of its 228 KB of shared memory (1 KB of which a block always
// takes), so that no two blocks of these kernels on one SM can want more
// columns than it has: an allocation then never waits, and clusters cannot
// wait for one another.
constexpr int mx_smem_floor(int cols) { return 228 * 1024 / 512 * cols - 1024; }

}  // namespace lutq
