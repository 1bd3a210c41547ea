// The product of two microscaled 4-bit matrices for many tokens: pairs of
// thread blocks (cta_group::2), tiles of 256 weight rows by up to 256 tokens.
//
// The arithmetic of lutq_mx_gemm.cu, laid out for a dense contraction.  Two
// blocks on neighbouring multiprocessors issue one MMA of 256 rows: each loads
// its own 128 weight rows and half of the tokens, so a 256 x 256 tile takes 64
// bytes a clock and multiprocessor from L2 at the tensor core's full rate (one
// block alone with 128 x 256 would take 96).  Scales of the tokens are loaded
// by both blocks, which each need all of them in tensor memory.
//
// A tile's sums fill 256 of the 512 columns.  The next tile's sums begin where
// the columns end that remain beside the scales, so that two tiles overlap by
// 64 (mxfp4) or 96 (nvfp4) columns: the epilogue empties those first, and the
// next tile's MMAs run while it empties the others.
//
// Gate and up: two sets of sums, and in mxfp4 the hidden values are quantized
// from the staged slice (a warp's 32 rows are one block), so that they pass
// through memory as 4-bit codes.  (nvfp4's row scale needs the whole row: those
// are written as bf16 and quantized by a launch of their own.)
//
// Few tokens: tiles of 512 weight rows where that saves a round (tall), or of
// 256 shared by K where they are fewer than pairs (split).
//
// Epilogue: eight warps, each on its own: 32 rows by 32 columns (tokens) at a
// time through shared memory and a tensor-map store, which also clips the tile
// to the output.
#include <algorithm>
#include <cstring>

#include "lutq_mx_gemm.cuh"
#include "lutq_sm100.cuh"

namespace lutq {

using namespace sm100;

constexpr uint64_t kPairWaitNs = 2000000000ull;
constexpr int kPairMaxStages = 10;
constexpr int kPairThreads = 64 + 256;
constexpr int kPairPrefetch = 10;    // chunks of weights brought to L2 ahead of the launch
constexpr int kPairTallTokens = 192;
constexpr int kPairTokenGroup = 16;  // token tiles that share a pass over the weights

// A pair's tile: plain, split by K over the pairs of a cluster, or tall (512
// weight rows).
enum PairTile { kPairPlain = 0, kPairSplit = 1, kPairTall = 2 };

template <int FMT, int MODE, int TILE>
struct PairCfg {
  static constexpr bool TALL = TILE == kPairTall;
  static constexpr int ND = MODE == kMxGateUp || TALL ? 2 : 1;  // sums of 256 weight rows
  static constexpr int ROWS = TALL ? 512 : 256;          // weight rows of a tile (of a matrix)
  static constexpr int NT = TALL ? kPairTallTokens : 256 / ND;  // tokens of a tile at most
  static constexpr int CH = mx_chunk_bytes(FMT);
  static constexpr int BLOCKS = CH / 512;
  static constexpr int A_BYTES = 128 * 128;
  // a stage for tiles of up to `width` columns: weights, half of the tokens, scales
  __host__ __device__ static constexpr int b_bytes(int width) { return width / 2 * 128; }
  __host__ __device__ static constexpr int stage(int width) {
    return ND * A_BYTES + b_bytes(width) + (ND + (width > kMxRowTile ? 2 : 1)) * CH;
  }
  static constexpr int SF_COLS = (ND + 2) * BLOCKS * 4;  // one set; two are kept
  // where the next tile's sums begin (tall: where these do), and the columns of both
  static constexpr int SECOND = TALL ? 0 : (512 - 2 * SF_COLS - 256) / 32 * 32;
  static_assert(!TALL || ND * NT + 2 * SF_COLS <= 512, "");
  static constexpr int SHARED_COLS = 256 - SECOND;
};

struct PairShared {
  uint64_t full[kPairMaxStages], empty[kPairMaxStages];
  uint64_t acc_full, acc_free, drain;
  uint64_t part_full;                    // split tiles
  uint32_t tmem;
  int abort;
  alignas(16) float row_scales[8][128];  // nvfp4: per epilogue warp, its tokens' of a tile
};

struct PairArgs {
  MxGemmArgs g;
  int token_tiles;    // plain: ceil(M / NT)
  int pairs;          // pairs of blocks in the launch
  int split;          // pairs that share a tile by K
  int tall;           // tiles of 512 weight rows
  int width;          // columns of the widest tile: what a stage has room for
  int slices;         // a warp's staged slices
  int tma_store;      // y by tensor-map stores (row pitch a multiple of 16 bytes)
};

// Columns of a tile with `valid` tokens: each block loads half of them, in
// boxes of 16.
__host__ __device__ __forceinline__ int pair_width(int valid) { return (valid + 31) / 32 * 32; }

__device__ __forceinline__ void pair_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_ns() - t0 > kPairWaitNs) return;
}

// Tile t of a launch: token tiles vary fastest (in groups), so that a weight
// tile is read from memory once per group and then from L2.  Tiles begin at
// multiples of 128 tokens (the height of a scale block), a last one is as wide
// as its tokens need.
template <int MODE, int ROWS>
struct PairTiles {
  static constexpr int nt = MODE == kMxGateUp ? 128 : 256;
  const int32_t* counts;
  int mtiles, experts, token_tiles, e = 0, e_tiles = 0;
  int64_t e_first = 0, tokens;
  __device__ PairTiles(const PairArgs& a, const int32_t* c)
      : counts(c), mtiles(int(mx_ceil(a.g.N, ROWS))), experts(a.g.experts),
        token_tiles(a.token_tiles), tokens(a.g.M) {
    if (MODE != kMxPlain) {
      tokens = counts[0];
      token_tiles = int(mx_ceil(tokens, nt));
      e_tiles = token_tiles * mtiles;
    }
  }
  __device__ bool at(int64_t t, int* expert, int* mt, int* m0, int* valid) {
    if constexpr (MODE != kMxPlain) {
      while (t >= e_first + e_tiles) {
        e_first += e_tiles;
        if (++e >= experts) {
          e = experts - 1;
          e_tiles = 0;
          return false;
        }
        tokens = counts[e];
        token_tiles = int(mx_ceil(tokens, nt));
        e_tiles = token_tiles * mtiles;
      }
      t -= e_first;
    } else {
      if (t >= int64_t(token_tiles) * mtiles) return false;
    }
    const int64_t per_group = int64_t(kPairTokenGroup) * mtiles;
    const int g = int(t / per_group), r = int(t - g * per_group);
    const int width = min(kPairTokenGroup, token_tiles - g * kPairTokenGroup);
    const int w = r / width;
    *expert = e;
    *mt = w;
    *m0 = (g * kPairTokenGroup + (r - w * width)) * nt;
    *valid = int(min(int64_t(nt), tokens - *m0));
    return true;
  }
};

// One value, rounded to the output type, into shared memory.
template <int DT>
__device__ __forceinline__ void stage1(uint32_t saddr, float v) {
  if constexpr (DT == LUTQ_FP32) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(saddr), "f"(v) : "memory");
  } else {
    const uint16_t h = DT == LUTQ_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v))
                                       : __half_as_ushort(__float2half_rn(v));
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(saddr), "h"(h) : "memory");
  }
}

// A slice of hidden values (bf16, 32 tokens x 32 rows in shared memory) to a
// block of codes and its scale byte for each token: lane t takes token t of
// the slice.  row: the tokens' first row in the packed buffer of a.M x a.N; n:
// the first of the 32 columns.
__device__ __forceinline__ bool pack_hidden(const MxGemmArgs& a, const uint8_t* slice, int64_t row,
                                            int n, int lane) {
  Raw8<LUTQ_BF16> raw[4];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    raw[j] = load_raw8<LUTQ_BF16>(slice, lane * 32 + 8 * j);
    m = max(m, max_raw8<LUTQ_BF16>(raw[j]));
  }
  const bool bad = m >= raw_inf<LUTQ_BF16>();
  const uint32_t scale = bad ? 0xFFu : e8m0_byte(max_bits_f32<LUTQ_BF16>(m));
  uint8_t* packed = static_cast<uint8_t*>(a.y);
  const int64_t r = row + lane;
  if (n < a.N) {
    uint32_t codes[4] = {0u, 0u, 0u, 0u};
    if (!bad) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float v[8];
        widen8<LUTQ_BF16>(raw[j], v);
        codes[j] = mx_codes8<LUTQ_MXFP4, LUTQ_BF16>(v, scale, 1.f, 1.f);
      }
    }
    *reinterpret_cast<uint4*>(packed + r * (a.N / 2) + n / 2) =
        make_uint4(codes[0], codes[1], codes[2], codes[3]);
  }
  // (columns behind the last are zeros: scale byte 0, as the layout wants)
  const int64_t chunk = (r / kMxRowTile) * mx_ceil(a.N, kMxChunk) + n / kMxChunk;
  const int block = n / 32 % 8;
  packed[mx_scale_off(a.M, a.N) + chunk * mx_chunk_bytes(LUTQ_MXFP4) + (block / 4) * 512 +
         int(r & 31) * 16 + int((r >> 5) & 3) * 4 + (block & 3)] = uint8_t(scale);
  return bad;
}

// SPLIT (plain products with few tiles): the pairs of a cluster share one tile
// by K, pair i taking chunks [C i / split, C (i+1) / split).  When a block's
// part is summed, its stages are free: the sums go there, and the pair that
// finishes a slice of 32 columns (slice s: pair s mod split) fetches and adds
// them in the order of the pairs.
//
// TALL (plain products of up to 192 tokens): two sums of 256 weight rows by all
// tokens, so that what a pair fetches of the tokens serves twice the weights.
template <int FMT, int MODE, int DT, int TILE>
__global__ void __launch_bounds__(kPairThreads, 1)
    mx_pair_kernel(const __grid_constant__ CUtensorMap tmap_a,
                   const __grid_constant__ CUtensorMap tmap_a2,
                   const __grid_constant__ CUtensorMap tmap_b,
                   const __grid_constant__ CUtensorMap tmap_b16,
                   const __grid_constant__ CUtensorMap tmap_sa,
                   const __grid_constant__ CUtensorMap tmap_sa2,
                   const __grid_constant__ CUtensorMap tmap_sb,
                   const __grid_constant__ CUtensorMap tmap_y, const PairArgs p) {
  using Cfg = PairCfg<FMT, MODE, TILE>;
  constexpr bool SPLIT = TILE == kPairSplit, TALL = Cfg::TALL;
  constexpr int ND = Cfg::ND, CH = Cfg::CH, BLOCKS = Cfg::BLOCKS, ROWS = Cfg::ROWS;
  constexpr int ES = DT == LUTQ_FP32 ? 4 : 2;
  constexpr int SLICE = 32 * 32 * ES;  // a staged slice: 32 tokens x a warp's 32 rows
  const MxGemmArgs& a = p.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int ST = a.stages;
  const uint32_t b_bytes = Cfg::b_bytes(p.width), stage_bytes = Cfg::stage(p.width);
  uint8_t* staging = smem + ST * stage_bytes;  // [8 warps][1 or 2] slices
  PairShared* sh = reinterpret_cast<PairShared*>(staging + 8 * p.slices * SLICE);
  int32_t* counts = reinterpret_cast<int32_t*>(sh + 1);
  const uint32_t sbase = smem_addr(smem);
  // warp-uniform for the compiler, too
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  // place in the pair, the pair in its cluster, the pair's first block
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, leader = crank & ~1u;
  const int split = SPLIT ? p.split : 1, part = SPLIT ? int(crank >> 1) : 0;
  const int c0 = SPLIT ? a.chunks * part / split : 0;
  const int c1 = SPLIT ? a.chunks * (part + 1) / split : a.chunks;
  volatile int* abort = &sh->abort;
  auto full = [&](int s) { return smem_addr(&sh->full[s]); };
  auto empty = [&](int s) { return smem_addr(&sh->empty[s]); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(smem_addr(&sh->acc_full), 1);
    mbar_init(smem_addr(&sh->acc_free), 16);  // eight warps of both blocks
    mbar_init(smem_addr(&sh->drain), 1);
    mbar_init(smem_addr(&sh->part_full), 8 * split);
    sh->abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(&sh->tmem), 512);
    tmem_relinquish_pair();
  }
  // While the work before this launch runs: the first chunks of the first tile
  // into L2.  (A prefetch reads nothing into the kernel; what that work may
  // still write, L2 has no stale copy of.)
  if (MODE == kMxPlain && warp == 0 && elect_one()) {
    const int64_t per_group = int64_t(kPairTokenGroup) * mx_ceil(a.N, ROWS);
    const int tile = int(blockIdx.x >> 1) / split;
    if (tile < per_group) {
      const int width = min(kPairTokenGroup, p.token_tiles);
      const int arow = tile / width * ROWS + int(rank) * 128;
      for (int c = c0; c < min(c1, c0 + kPairPrefetch / (ROWS / 256)); ++c) {
        tma_3d_prefetch(&tmap_a, c * 128, arow, 0);
        if (TALL) tma_3d_prefetch(&tmap_a, c * 128, arow + 256, 0);
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (MODE != kMxPlain) {
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
      counts[e] = a.counts[e];
      counts[a.experts + e] = a.bases[e];
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem, 0);
  const int64_t first = (blockIdx.x >> 1) / split, step = p.pairs / split;
  const uint32_t full0 = cluster_map(full(0), leader);  // the pair's first block's barriers
  PairTiles<MODE, ROWS> tiles(p, counts);
  int expert, mt, m0, valid;

  if (warp == 0) {
    // ------------------------------------------------------------ copies (both blocks)
    int s = 0;
    uint32_t ph = 1;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t t = first; ok && tiles.at(t, &expert, &mt, &m0, &valid); t += step) {
      const int row0 = MODE == kMxPlain ? m0 : counts[a.experts + expert] + m0;
      const int arow = mt * ROWS + int(rank) * 128;
      const int arow2 = arow + (TALL ? 256 : 0);  // the second sums' rows
      const int half = pair_width(valid) / 2;
      const int brow = row0 + int(rank) * half;
      // the token scales of one or two tiles of 128 rows
      const int sb_tiles = half > kMxRowTile / 2 ? 2 : 1;
      const uint32_t bytes = 2u * uint32_t(ND * (Cfg::A_BYTES + CH) + half * 128 + sb_tiles * CH);
      const int sa_row = (arow / 128) * a.chunks * (CH / 1024);
      const int sa_row2 = (arow2 / 128) * a.chunks * (CH / 1024);
      const int sb_row = (row0 / kMxRowTile) * a.chunks * (CH / 1024);
      for (int c = c0; c < c1; ++c) {
        ok = mbar_wait(empty(s), ph, abort, kPairWaitNs);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const uint32_t st = sbase + s * stage_bytes;
        const uint32_t sb = st + ND * Cfg::A_BYTES, sf = sb + b_bytes;
        const uint32_t bar = full0 + 8 * s;
        const int sc = c * (CH / 1024);
        if (elect_one()) {
          if (rank == 0) mbar_expect_tx(full(s), bytes);
          tma_3d_g2s_pair(st, &tmap_a, c * 128, arow, expert, bar);
          if (ND == 2) tma_3d_g2s_pair(st + Cfg::A_BYTES, &tmap_a2, c * 128, arow2, expert, bar);
          if (2 * half == p.width) {
            tma_3d_g2s_pair(sb, &tmap_b, c * 128, brow, 0, bar);
          } else {
            for (int i = 0; i < half; i += 16)
              tma_3d_g2s_pair(sb + i * 128, &tmap_b16, c * 128, brow + i, 0, bar);
          }
          tma_3d_g2s_pair(sf, &tmap_sa, 0, sa_row + sc, expert, bar);
          if (ND == 2) tma_3d_g2s_pair(sf + CH, &tmap_sa2, 0, sa_row2 + sc, expert, bar);
          tma_3d_g2s_pair(sf + ND * CH, &tmap_sb, 0, sb_row + sc, 0, bar);
          if (sb_tiles == 2)
            tma_3d_g2s_pair(sf + (ND + 1) * CH, &tmap_sb, 0,
                            sb_row + a.chunks * (CH / 1024) + sc, 0, bar);
        }
        __syncwarp();
        ++issued;
        if (++s == ST) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (__any_sync(0xffffffffu, *abort) && rank == 0) {
      // let both blocks' copies land before either leaves
      const int64_t n = issued < ST ? issued : ST;
      for (int64_t i = issued - n; i < issued; ++i)
        pair_drain(full(int(i % ST)), uint32_t(i / ST) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs (first block)
    if (rank == 0) {
      constexpr bool E8 = FMT == LUTQ_MXFP4;
      int s = 0, it = 0, n = 0;
      uint32_t ph = 0;
      bool ok = true, any = false;
      for (int64_t t = first; ok && tiles.at(t, &expert, &mt, &m0, &valid); t += step, ++n) {
        // the tile before must have left the shared columns
        if (n > 0) ok = mbar_wait_cluster(smem_addr(&sh->acc_free), uint32_t(n - 1) & 1u, abort,
                                          kPairWaitNs);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t d = tmem + uint32_t((n & 1) * Cfg::SECOND);
        const int width = pair_width(valid), sb_tiles = width > kMxRowTile ? 2 : 1;
        const uint32_t idesc = idesc_e2m1(256, width, E8, 0);
        const uint32_t id2 = idesc_e2m1(0, 0, false, 2);  // the scale bytes 2 and 3
        for (int c = c0; c < c1; ++c, ++it) {
          ok = mbar_wait(full(s), ph, abort, kPairWaitNs);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          tc_fence_after();
          const uint32_t st = desc_lo(sbase + s * stage_bytes);
          const uint32_t bl = st + ((ND * Cfg::A_BYTES) >> 4);
          const uint32_t sf = bl + (b_bytes >> 4);
          const uint32_t sf_tmem = tmem + 512u - uint32_t(2 - (it & 1)) * Cfg::SF_COLS;
          const uint32_t sb_tmem = sf_tmem + ND * BLOCKS * 4;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < ND * BLOCKS; ++i) tmem_cp_scales_pair(sf_tmem + 4 * i, sf + 32 * i);
            // the tokens' blocks side by side: [block][row tile]
#pragma unroll
            for (int i = 0; i < BLOCKS; ++i)
              tmem_cp_scales_pair(sb_tmem + 8 * i, sf + ((ND * CH) >> 4) + 32 * i);
            if (sb_tiles == 2) {
#pragma unroll
              for (int i = 0; i < BLOCKS; ++i)
                tmem_cp_scales_pair(sb_tmem + 8 * i + 4, sf + (((ND + 1) * CH) >> 4) + 32 * i);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // mxfp4: a block holds the scales of two MMAs, nvfp4: of one
              const int blk = E8 ? j >> 1 : j;
#pragma unroll
              for (int w = 0; w < ND; ++w)
                mma_e2m1_pair<!E8>(d + w * Cfg::NT, st + ((w * Cfg::A_BYTES) >> 4) + 2 * j,
                                   bl + 2 * j, E8 && (j & 1) ? idesc | id2 : idesc,
                                   sf_tmem + 4 * (w * BLOCKS + blk), sb_tmem + 8 * blk,
                                   (c > c0 || j > 0) ? 1u : 0u);
            }
            mma_commit_pair(empty(s), 3u << leader);
          }
          __syncwarp();
          any = true;
          if (++s == ST) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        if (elect_one()) mma_commit_pair(smem_addr(&sh->acc_full), 3u << leader);
        __syncwarp();
      }
      if (__any_sync(0xffffffffu, *abort) && any) {
        if (elect_one()) mma_commit_pair(smem_addr(&sh->drain), 3u << leader);
        __syncwarp();
        pair_drain(smem_addr(&sh->drain), 0);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, group = (warp - 2) >> 2;  // four warps cover the 128 lanes
    uint8_t* stage0 = staging + (warp - 2) * p.slices * SLICE;
    float* gbs = sh->row_scales[warp - 2];  // nvfp4: the row scales of this warp's tokens
    int n = 0, slot = 0;
    bool ok = true, bad = false;
    // slices of 32 columns, this group's are column(n, 0), column(n, 1), ...:
    // those that the next tile's sums share come first, the last ones of an
    // even tile (columns SECOND..255) and the first ones of an odd tile.
    // (With two sets the shared columns are the end of the second or the
    // beginning of the first.)
    constexpr int NS = Cfg::NT / 32, OWN = NS / 2;
    auto column_of = [&](int tile, int i) {
      const int sl = group + 2 * i;
      return 32 * (!TALL && (tile & 1) == 0 ? NS - 1 - sl : sl);
    };
    // nvfp4: a tile's row scales are fetched while the tile before is worked on
    float ga[2] = {1.f, 1.f}, ga_next[2] = {1.f, 1.f}, gb_next[OWN];
    auto fetch = [&](int tile) {
      const int r = mt * ROWS + int(rank) * 128 + quarter * 32 + lane;
      const int64_t first_token = MODE == kMxPlain ? m0 : counts[a.experts + expert] + m0;
#pragma unroll
      for (int w = 0; w < ND; ++w) {
        const int rw = r + (TALL ? 256 * w : 0);
        if (rw < a.N)
          ga_next[w] = *reinterpret_cast<const float*>(
              reinterpret_cast<const uint8_t*>(a.a_rows[w]) + int64_t(expert) * a.a_stride +
              int64_t(rw) * 4);
      }
#pragma unroll
      for (int i = 0; i < OWN; ++i)
        if (column_of(tile, i) < valid)
          gb_next[i] = a.b_rows[first_token + column_of(tile, i) + lane];
    };
    bool more = tiles.at(first, &expert, &mt, &m0, &valid);
    if (FMT == LUTQ_NVFP4 && more) fetch(0);
    for (int64_t t = first; more; t += step, ++n) {
      const int row0 = mt * ROWS + int(rank) * 128 + quarter * 32 + lane;
      const int tokens = valid;
      const int64_t token0 = MODE == kMxPlain ? m0 : counts[a.experts + expert] + m0;
      const uint32_t d = tmem + (uint32_t(quarter * 32) << 16) + uint32_t((n & 1) * Cfg::SECOND);
      auto column = [&](int i) { return column_of(n, i); };
      if (FMT == LUTQ_NVFP4) {
#pragma unroll
        for (int w = 0; w < ND; ++w) ga[w] = ga_next[w];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < OWN; ++i) gbs[32 * i + lane] = gb_next[i];
        __syncwarp();
      }
      more = tiles.at(t + step, &expert, &mt, &m0, &valid);  // the tile after this one
      ok = mbar_wait(smem_addr(&sh->acc_full), uint32_t(n) & 1u, abort, kPairWaitNs);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc_fence_after();

      // one slice: scale, round, stage, store (SETS: of one or of two sums)
      constexpr int SETS = TALL ? 1 : ND;
      auto finish = [&](int c, const float* gbc, uint32_t (&v)[SETS][32], int set) {
        const int row = row0 + 256 * set;
        const float ga0 = TALL && set == 1 ? ga[1] : ga[0];
        uint8_t* stg = stage0 + slot * SLICE;
        const uint32_t sta = smem_addr(stg) + lane * ES;
        float4 s4[8];  // (all before the first store: it would order the loads)
        if (FMT == LUTQ_NVFP4) {
#pragma unroll
          for (int q = 0; q < 8; ++q) s4[q] = reinterpret_cast<const float4*>(gbc)[q];
        }
        // the store that read this buffer last must be done
        if (lane == 0) {
          if (p.slices == 2) bulk_wait_read<1>();
          else bulk_wait_read<0>();
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float f = __uint_as_float(v[0][j]), u = __uint_as_float(v[SETS - 1][j]);
          if (FMT == LUTQ_NVFP4) {
            const float4 q4 = s4[j / 4];
            const float gb = j % 4 == 0 ? q4.x : j % 4 == 1 ? q4.y : j % 4 == 2 ? q4.z : q4.w;
            f = f * ga0 * gb;
            if (SETS == 2) u = u * ga[1] * gb;
          }
          if (SETS == 2) f = silu_mul(f, u);
          stage1<DT>(sta + j * 32 * ES, f);
        }
        if (MODE == kMxGateUp && FMT == LUTQ_MXFP4) {
          // straight into the down product's operand
          __syncwarp();
          const bool nan = pack_hidden(a, stg, token0 + c, row - lane, lane);
          bad |= nan && c + lane < tokens;
        } else if (p.tma_store) {
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            if (row < a.N) tma_2d_s2g(&tmap_y, row, int(token0) + c, smem_addr(stg));
            bulk_commit();  // (a group a slice: the wait above counts them)
          }
        } else {
          // rows that no 16-byte copy can write: each warp its own lanes
          __syncwarp();
          if (row < a.N)
            for (int j = 0; j < 32 && c + j < tokens; ++j) {
              const int64_t at = (token0 + c + j) * a.N + row;
              if (ES == 4)
                static_cast<uint32_t*>(a.y)[at] =
                    reinterpret_cast<const uint32_t*>(stg)[j * 32 + lane];
              else
                static_cast<uint16_t*>(a.y)[at] =
                    reinterpret_cast<const uint16_t*>(stg)[j * 32 + lane];
            }
        }
        slot ^= p.slices - 1;
      };
      auto load = [&](int i, uint32_t (&v)[SETS][32]) {
        if (column(i) < tokens) {
#pragma unroll
          for (int w = 0; w < SETS; ++w) tmem_ld_32x32b_x32(d + w * Cfg::NT + column(i), v[w]);
        }
      };
      if constexpr (SPLIT) {
        // (one tile a cluster) the sums into the block's stages, which hold
        // nothing any more, [column][row]: the block of the same place in the
        // pair that finishes a slice fetches it from there
        float* mine = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
        uint32_t v[1][32];
#pragma unroll 1
        for (int c = 32 * group; c < tokens; c += 64) {
          tmem_ld_32x32b_x32(d + c, v[0]);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) mine[(c + j) * 128] = __uint_as_float(v[0][j]);
        }
        __syncwarp();
        if (lane < split)
          cluster_arrive(cluster_map(smem_addr(&sh->part_full), 2u * lane + rank));
        ok = mbar_wait_cluster(smem_addr(&sh->part_full), 0, abort, kPairWaitNs);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
#pragma unroll 1
        for (int k = group; 32 * (k * split + part) < tokens; k += 2) {
          const int c = 32 * (k * split + part);
          float sum[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[j] = 0.f;
#pragma unroll 1
          for (int q = 0; q < split; ++q) {
            const uint32_t from = cluster_map(smem_addr(mine + c * 128), 2u * uint32_t(q) + rank);
            float u[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) u[j] = cluster_ld_f32(from + j * 512);
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[j] += u[j];
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[0][j] = __float_as_uint(sum[j]);
          if (FMT == LUTQ_NVFP4) {
            __syncwarp();
            gbs[lane] = a.b_rows[token0 + c + lane];
            __syncwarp();
          }
          finish(c, gbs, v, 0);
        }
        break;
      }
      if constexpr (TALL) {
        uint32_t v[1][32];
        for (int set = 0; set < 2; ++set) {
#pragma unroll 1
          for (int i = 0; column(i) < tokens && i < OWN; ++i) {
            tmem_ld_32x32b_x32(d + set * Cfg::NT + column(i), v[0]);
            tmem_wait_ld();
            finish(column(i), gbs + 32 * i, v, set);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cluster_arrive(cluster_map(smem_addr(&sh->acc_free), leader));
        if (FMT == LUTQ_NVFP4 && more) fetch(n + 1);
        continue;
      }
      // two slices in registers; the shared columns are among the first two of
      // each group, so the next tile's MMAs wait for no more than these loads
      static_assert(TALL || (Cfg::SHARED_COLS <= 128 && OWN >= 2), "");
      uint32_t va[SETS][32], vb[SETS][32];
      load(0, va);
      load(1, vb);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) cluster_arrive(cluster_map(smem_addr(&sh->acc_free), leader));
      if (FMT == LUTQ_NVFP4 && more) fetch(n + 1);
#pragma unroll
      for (int i = 0; i < OWN; i += 2) {
        if (i > 0) {
          load(i, va);
          load(i + 1, vb);
          tmem_wait_ld();
        }
        if (column(i) < tokens) finish(column(i), gbs + 32 * i, va, 0);
        if (column(i + 1) < tokens) finish(column(i + 1), gbs + 32 * (i + 1), vb, 0);
      }
    }
    if (lane == 0) bulk_wait<0>();
    if (bad) report(a.dev_status, LUTQ_ERR_NONFINITE);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort) report(a.dev_status, LUTQ_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ host side

template <int FMT, int MODE, int DT, int TILE>
static cudaError_t launch_one(const MxPairMaps& m, PairArgs p, cudaStream_t stream) {
  using Cfg = PairCfg<FMT, MODE, TILE>;
  constexpr int SLICE = 32 * 32 * (DT == LUTQ_FP32 ? 4 : 2);
  constexpr int smem = 227 * 1024;  // all of it: the block holds all of tensor memory
  auto stages = [&](int slices) {
    const int fixed = 1024 + 8 * slices * SLICE + int(sizeof(PairShared)) +
                      (MODE != kMxPlain ? 8 * p.g.experts : 0);
    return std::min(kPairMaxStages, (smem - fixed) / Cfg::stage(p.width));
  };
  // Tall tiles: a second staged slice where it does not cost a stage.  28672 x
  // 8192, one slice / two, us: nvfp4, 133 tokens 31.2 / 32.8, 192 (where one
  // gives no stage more) 35.3 / 35.1; mxfp4, 192 tokens 30.2 / 31.3, 133 (no
  // stage more) 28.4 / 27.9; alike at 57344 x 8192, 24576 x 4096, 20480 x 5120.
  if (Cfg::TALL) p.slices = stages(1) > stages(2) ? 1 : 2;
  p.g.stages = stages(p.slices);
  // A split tile's sums, 512 bytes a column, fit in four stages of any width:
  // 4 (16 KB + 64 width) >= 512 width for up to 256 columns.
  static_assert(TILE != kPairSplit ||
                    (smem - 1024 - 8 * SLICE - int(sizeof(PairShared))) / Cfg::stage(256) >= 4,
                "");
  auto kernel = mx_pair_kernel<FMT, MODE, DT, TILE>;
  static bool granted[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!granted[dev]) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    granted[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(2 * p.pairs));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {unsigned(2 * p.split), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, m.a[0], m.a[1], m.b, m.b16, m.sa[0], m.sa[1], m.sb, m.y,
                            p);
}

template <int FMT, int DT>
static cudaError_t launch_plain(const MxPairMaps& m, const PairArgs& p, cudaStream_t stream) {
  if (p.tall) return launch_one<FMT, kMxPlain, DT, kPairTall>(m, p, stream);
  return p.split > 1 ? launch_one<FMT, kMxPlain, DT, kPairSplit>(m, p, stream)
                     : launch_one<FMT, kMxPlain, DT, kPairPlain>(m, p, stream);
}

template <int FMT>
static cudaError_t launch_fmt(const MxPairMaps& m, const PairArgs& p, int mode,
                              cudaStream_t stream) {
  if (mode == kMxGateUp) return launch_one<FMT, kMxGateUp, LUTQ_BF16, kPairPlain>(m, p, stream);
  if (mode == kMxDown) return launch_one<FMT, kMxDown, LUTQ_FP32, kPairPlain>(m, p, stream);
  if (p.g.y_dtype == LUTQ_BF16) return launch_plain<FMT, LUTQ_BF16>(m, p, stream);
  if (p.g.y_dtype == LUTQ_FP16) return launch_plain<FMT, LUTQ_FP16>(m, p, stream);
  return launch_plain<FMT, LUTQ_FP32>(m, p, stream);
}

// How a plain product (lutq_mx_gemm) is divided: see lutq_mx_gemm_plan.
MxPairPlan mx_pair_plan(int64_t M, int64_t N, int64_t K, int fmt, int num_sms) {
  MxPairPlan p = {};
  p.width = pair_width(int(std::min<int64_t>(M, 256)));
  p.tiles = mx_ceil(N, 256) * mx_ceil(M, 256);
  const int chunks = int(mx_ceil(K, kMxChunk)), slots = std::max(1, num_sms / 2);
  // Split tiles by K while that gives idle pairs work and saves more chunks (0.3 us
  // each) than the exchange costs (1.5 us for 32 columns, 3 for 256; 4096 x 14336
  // at 512 tokens 23.6 -> 20.3 us, 512 x 14336 at 128 tokens 22.6 -> 13.0).
  // Clusters of eight blocks that fill their multiprocessors leave many unused:
  // sixteen of them ran in two waves.  (Every tile needs pairs of its own.)
  const int per = p.tiles <= 16 && M <= 128 ? 8 : 12;
  p.split = 1;
  if (p.tiles <= 32 && 2 * p.tiles <= slots && chunks >= 2 * per)
    p.split = p.tiles <= 8 && 4 * p.tiles <= slots && chunks >= 4 * per ? 4 : 2;
  // Tall tiles where they save a round: what bounds a tile is what its pair
  // fetches, 85 GB/s a multiprocessor.  28672 x 8192 in nvfp4 at 133 tokens: 2
  // rounds of 32 KB a chunk and block take 35.2 us, 1 of 50 KB 30.5; at 17
  // tokens 2 of 22 KB 27.8, 1 of 40 KB 24.9.
  if (p.split == 1 && p.width <= kPairTallTokens) {
    auto fetched = [&](int nd) {
      const int a_bytes = 128 * 128 + mx_chunk_bytes(fmt);
      const int b_bytes = p.width * 64 + (p.width > kMxRowTile ? 2 : 1) * mx_chunk_bytes(fmt);
      return mx_ceil(mx_ceil(N, 256 * nd), slots) * (nd * a_bytes + b_bytes);
    };
    p.tall = fetched(2) < fetched(1);
    if (p.tall) p.tiles = mx_ceil(N, 512);
  }
  p.pairs = int(std::max<int64_t>(1, std::min<int64_t>(p.tiles, slots / p.split))) * p.split;
  // Slices are staged while the next tile's MMAs run, two a warp; where there
  // is no next tile, one, and a stage more instead (133 tokens x 9472 x 8192 in
  // nvfp4 16.2 -> 15.7 us, in mxfp4 14.6 -> 14.3).  (Tall: see launch_one.)
  p.slices = p.tiles * p.split <= p.pairs ? 1 : 2;
  return p;
}

cudaError_t launch_mx_pair(const MxGemmArgs& g, const void* weights, const void* weights2,
                           int64_t w_bytes, const void* tokens, int64_t token_rows, int fmt,
                           int mode, int64_t tiles, int num_sms, cudaStream_t stream) {
  MxPairMaps m;
  std::memset(&m, 0, sizeof(m));
  const int64_t batch = std::max(1, g.experts);
  const void* w[2] = {weights, weights2};
  cudaError_t err;
  const int nd = mode == kMxGateUp ? 2 : 1;
  for (int i = 0; i < nd; ++i) {
    if ((err = make_mx_map(&m.a[i], w[i], g.N, g.K, batch, w_bytes, 128)) != cudaSuccess)
      return err;
    if ((err = make_mx_scale_map(&m.sa[i], w[i], g.N, g.K, batch, w_bytes, fmt)) != cudaSuccess)
      return err;
  }
  const int64_t t_bytes = mx_bytes(token_rows, g.K, fmt);
  const int nt = mode == kMxGateUp ? 128 : 256;
  PairArgs p = {};
  p.g = g;
  p.token_tiles = int(mx_ceil(g.M, nt));
  if (mode == kMxPlain) {
    // Few tokens leave room for more stages, which come at the latency of memory
    // (9472 x 8192 in nvfp4, 17 tokens: 8 stages for 4, 15.2 -> 13.5 us).
    const MxPairPlan plan = mx_pair_plan(g.M, g.N, g.K, fmt, num_sms);
    p.width = plan.width;
    p.split = plan.split;
    p.tall = plan.tall;
    p.pairs = plan.pairs;
    p.slices = plan.slices;
    if (p.tall) {
      m.a[1] = m.a[0];
      m.sa[1] = m.sa[0];
    }
  } else {
    p.width = nt;
    p.split = 1;
    p.pairs = int(std::max<int64_t>(1, std::min<int64_t>(tiles, num_sms / 2)));
    p.slices = 2;
  }
  if ((err = make_mx_map(&m.b, tokens, token_rows, g.K, 1, t_bytes, p.width / 2)) != cudaSuccess)
    return err;
  if ((err = make_mx_map(&m.b16, tokens, token_rows, g.K, 1, t_bytes, 16)) != cudaSuccess)
    return err;
  if ((err = make_mx_scale_map(&m.sb, tokens, token_rows, g.K, 1, t_bytes, fmt)) != cudaSuccess)
    return err;
  const int dt = mode == kMxGateUp ? int(LUTQ_BF16) : g.y_dtype;
  p.tma_store = (g.N * (dt == LUTQ_FP32 ? 4 : 2)) % 16 == 0 &&
                !(mode == kMxGateUp && fmt == LUTQ_MXFP4);  // (quantized instead)
  if (p.tma_store) {
    if ((err = make_mx_out_map(&m.y, g.y, g.M, g.N, dt)) != cudaSuccess) return err;
  }
  return fmt == LUTQ_MXFP4 ? launch_fmt<LUTQ_MXFP4>(m, p, mode, stream)
                           : launch_fmt<LUTQ_NVFP4>(m, p, mode, stream);
}

}  // namespace lutq
