// The experts' products of microscaled 4-bit matrices for a few to some dozen
// tokens an expert: packed tokens, laid out by expert, with each expert's
// weights (fewer tokens: lutq_mx_small.cu, more: lutq_mx_pair.cu).
//
// The tensor core multiplies the codes and applies both scales itself
// (tcgen05.mma with block scales), so nothing is dequantized: the kernel only
// moves bytes, and is bound by the weights'.  A tile is 128 rows of a weight
// matrix (the lanes of tensor memory) by NT tokens (its columns); taking the
// weights as the first operand keeps the tile narrow for few tokens, and a
// warp's 32 lanes are 32 neighbouring outputs of one token.  A stage is 256
// elements of K: 128 bytes a row of each operand by tensor-map copies with the
// 128-byte swizzle, the scale chunks by bulk copies, and per stage four MMAs of
// 64 elements.  Scale blocks go from shared memory to tensor memory with one
// copy instruction each, ordered before the MMAs.
//
// A cluster of `split` blocks shares a tile by K where tiles are few: block r
// takes chunks [C r / split, C (r+1) / split), and each block adds up its share
// of the columns over the cluster through distributed shared memory, in rank
// order, so that results do not depend on timing and no workspace is needed.
//
// Warps: 0 copies, 1 issues, 2..5 read tensor memory and write.
#include "lutq_mx_gemm.cuh"

#include <algorithm>
#include <cstring>

#include "lutq_sm100.cuh"

namespace lutq {

using namespace sm100;

constexpr uint64_t kMxWaitNs = 2000000000ull;
constexpr int kMxMaxStages = 8;

template <int FMT, int NT, int MODE>
struct MxCfg {
  static constexpr int ND = MODE == kMxGateUp ? 2 : 1;     // weight matrices a tile multiplies
  static constexpr int CH = mx_chunk_bytes(FMT);
  static constexpr int BLOCKS = CH / 512;                  // scale blocks per chunk
  static constexpr int A_BYTES = 128 * 128, B_BYTES = NT * 128;
  static constexpr int STAGE = ND * A_BYTES + B_BYTES + (ND + 1) * CH;
  static constexpr int SUMS = ND * NT * 128 * 4;           // partial sums of a split tile
  // tensor memory: accumulators (two sets where they fit), then two sets of scales
  static constexpr int SF_COLS = 2 * (ND + 1) * BLOCKS * 4;
  static constexpr int ACC = 2 * ND * NT + SF_COLS <= 512 ? 2 : 1;
  static constexpr int COLS = ACC * ND * NT + SF_COLS;
  static constexpr int TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
};

// Shared memory behind the stages: barriers, flags, small tables.
struct MxShared {
  uint64_t full[kMxMaxStages], empty[kMxMaxStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t part_full, part_empty, drain;
  uint32_t tmem;
  int abort;
};

// A tile begins at a multiple of 128 rows of the packed tokens, the height of a
// scale block (an expert's n-th tile of nt tokens at its row 128 n), so that
// its scales begin at the first column and lane of a block: the MMA faults on
// others ("misaligned address" with scales one column on).
//
// Walks the tiles t = first, first + step, ... of a launch, each expert's in turn.
struct MxTiles {
  const int32_t* counts;
  int mtiles, nt, experts, e = 0, e_tiles;
  int64_t e_first = 0;
  __device__ MxTiles(const MxGemmArgs& a, int nt_, const int32_t* counts_)
      : counts(counts_), mtiles(a.mtiles), nt(nt_), experts(a.experts),
        e_tiles(int(mx_ceil(counts_[0], nt_)) * a.mtiles) {}
  // false: no tile t; else its expert, row tile, first row of tokens and tokens
  __device__ bool at(int64_t t, int* expert, int* mt, int* m0, int* valid) {
    while (t >= e_first + e_tiles) {
      e_first += e_tiles;
      if (++e >= experts) {
        e = experts - 1;
        e_tiles = 0;
        return false;
      }
      e_tiles = int(mx_ceil(counts[e], nt)) * mtiles;
    }
    const int i = int(t - e_first), n = i / mtiles;
    *expert = e;
    *mt = i - n * mtiles;
    *m0 = n * 128;
    *valid = min(nt, counts[e] - n * nt);
    return true;
  }
};

// Bounded wait for work already in flight, whatever the abort flag says.
__device__ __forceinline__ void mx_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_ns() - t0 > kMxWaitNs) return;
}

template <int FMT, int NT, int MODE>
__global__ void __launch_bounds__(192)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmap_a,
                   const __grid_constant__ CUtensorMap tmap_a2,
                   const __grid_constant__ CUtensorMap tmap_b,
                   const __grid_constant__ CUtensorMap tmap_b16, const MxGemmArgs a, int split) {
  using Cfg = MxCfg<FMT, NT, MODE>;
  constexpr int ND = Cfg::ND, CH = Cfg::CH, BLOCKS = Cfg::BLOCKS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int ST = a.stages;
  float* sums = reinterpret_cast<float*>(smem + ST * Cfg::STAGE);
  MxShared* sh = reinterpret_cast<MxShared*>(smem + ST * Cfg::STAGE + (split > 1 ? Cfg::SUMS : 0));
  int32_t* counts = reinterpret_cast<int32_t*>(sh + 1);  // experts' row counts, then bases
  const uint32_t sbase = smem_addr(smem);
  // warp-uniform for the compiler, too
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  volatile int* abort = &sh->abort;
  auto full = [&](int s) { return smem_addr(&sh->full[s]); };
  auto empty = [&](int s) { return smem_addr(&sh->empty[s]); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&sh->acc_full[b]), 1);
      mbar_init(smem_addr(&sh->acc_empty[b]), 4);
    }
    mbar_init(smem_addr(&sh->part_full), 4 * split);
    mbar_init(smem_addr(&sh->part_empty), 4 * split);
    mbar_init(smem_addr(&sh->drain), 1);
    sh->abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&sh->tmem), Cfg::TMEM);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
    counts[e] = a.counts[e];
    counts[a.experts + e] = a.bases[e];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (split > 1) cluster_sync_all();  // every block's barriers are set up
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem, 0);
  const uint32_t rank = split > 1 ? cluster_ctarank() : 0u;
  const int64_t first = blockIdx.x / split, step = gridDim.x / split;
  const int c0 = int(int64_t(a.chunks) * rank / split);
  const int c1 = int(int64_t(a.chunks) * (rank + 1) / split);
  MxTiles tiles(a, NT, counts);
  int expert, mt, m0, valid;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    int s = 0;
    uint32_t ph = 1;
    int64_t issued = 0;
    bool ok = true;
    for (int64_t t = first; ok && tiles.at(t, &expert, &mt, &m0, &valid); t += step) {
      const int row0 = counts[a.experts + expert] + m0;
      const int width = (valid + 15) / 16 * 16;  // columns: in boxes of 16 tokens
      const int64_t a_off = int64_t(expert) * a.a_stride + int64_t(mt) * a.chunks * CH;
      const uint8_t* as = a.a_scales[0] + a_off;
      const uint8_t* as2 = a.a_scales[1] + a_off;
      const uint8_t* bs = a.b_scales + int64_t(row0 / kMxRowTile) * a.chunks * CH;
      const uint32_t bytes = ND * (Cfg::A_BYTES + CH) + width * 128 + CH;
      for (int c = c0; c < c1; ++c) {
        ok = mbar_wait(empty(s), ph, abort, kMxWaitNs);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        const uint32_t st = sbase + s * Cfg::STAGE;
        const uint32_t sb = st + ND * Cfg::A_BYTES, sf = sb + Cfg::B_BYTES;
        if (elect_one()) {
          mbar_expect_tx(full(s), bytes);
          tma_3d_g2s(st, &tmap_a, c * 128, mt * 128, expert, full(s));
          if (ND == 2) tma_3d_g2s(st + Cfg::A_BYTES, &tmap_a2, c * 128, mt * 128, expert, full(s));
          bulk_g2s(sf, as + int64_t(c) * CH, CH, full(s));
          if (ND == 2) bulk_g2s(sf + CH, as2 + int64_t(c) * CH, CH, full(s));
          if (width == NT) {
            tma_3d_g2s(sb, &tmap_b, c * 128, row0, 0, full(s));
          } else {
            for (int i = 0; i < width; i += 16)
              tma_3d_g2s(sb + i * 128, &tmap_b16, c * 128, row0 + i, 0, full(s));
          }
          bulk_g2s(sf + ND * CH, bs + int64_t(c) * CH, CH, full(s));
        }
        __syncwarp();
        ++issued;
        if (++s == ST) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // given up: the copies in flight must land before the block may exit
    if (__any_sync(0xffffffffu, *abort)) {
      const int64_t n = issued < ST ? issued : ST;
      for (int64_t i = issued - n; i < issued; ++i)
        mx_drain(full(int(i % ST)), uint32_t(i / ST) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    constexpr bool E8 = FMT == LUTQ_MXFP4;
    int s = 0, it = 0, n = 0;
    uint32_t ph = 0;
    bool ok = true, any = false;
    for (int64_t t = first; ok && tiles.at(t, &expert, &mt, &m0, &valid); t += step, ++n) {
      const int b = Cfg::ACC == 2 ? n & 1 : 0;
      const uint32_t use = uint32_t(Cfg::ACC == 2 ? n >> 1 : n);
      ok = mbar_wait(smem_addr(&sh->acc_empty[b]), (use & 1u) ^ 1u, abort, kMxWaitNs);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      tc_fence_after();
      const uint32_t d = tmem + uint32_t(b * ND * NT);
      const int width = (valid + 15) / 16 * 16;
      const uint32_t idesc = idesc_e2m1(128, width, E8, 0);
      const uint32_t id2 = idesc_e2m1(0, 0, false, 2);  // the scale bytes 2 and 3
      for (int c = c0; c < c1; ++c, ++it) {
        ok = mbar_wait(full(s), ph, abort, kMxWaitNs);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t st = desc_lo(sbase + s * Cfg::STAGE);
        const uint32_t bl = st + ((ND * Cfg::A_BYTES) >> 4);
        const uint32_t sf = bl + (Cfg::B_BYTES >> 4);
        const uint32_t sf_tmem =
            tmem + uint32_t(Cfg::ACC * ND * NT + (it & 1) * (Cfg::SF_COLS / 2));
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < (ND + 1) * BLOCKS; ++i) tmem_cp_scales(sf_tmem + 4 * i, sf + 32 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // mxfp4: a block holds the scales of two MMAs, nvfp4: of one
            const int blk = E8 ? j >> 1 : j;
#pragma unroll
            for (int w = 0; w < ND; ++w)
              mma_e2m1_ss<!E8>(d + w * NT, st + ((w * Cfg::A_BYTES) >> 4) + 2 * j, bl + 2 * j,
                               E8 && (j & 1) ? idesc | id2 : idesc,
                               sf_tmem + 4 * (w * BLOCKS + blk),
                               sf_tmem + 4 * (ND * BLOCKS + blk), (c > c0 || j > 0) ? 1u : 0u);
          }
          mma_commit(empty(s));
        }
        __syncwarp();
        any = true;
        if (++s == ST) {
          s = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) mma_commit(smem_addr(&sh->acc_full[b]));
      __syncwarp();
    }
    if (__any_sync(0xffffffffu, *abort) && any) {
      if (elect_one()) mma_commit(smem_addr(&sh->drain));
      __syncwarp();
      mx_drain(smem_addr(&sh->drain), 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    int n = 0;
    bool ok = true;
    // (NT / split) columns of the tile are this block's to sum and write
    const int own = NT / split;
    for (int64_t t = first; ok && tiles.at(t, &expert, &mt, &m0, &valid); t += step, ++n) {
      const int b = Cfg::ACC == 2 ? n & 1 : 0;
      const uint32_t use = uint32_t(Cfg::ACC == 2 ? n >> 1 : n);
      ok = mbar_wait(smem_addr(&sh->acc_full[b]), use & 1u, abort, kMxWaitNs);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int64_t row = int64_t(mt) * 128 + quarter * 32 + lane;
      const int64_t token0 = counts[a.experts + expert] + m0;
      const uint32_t d = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(b * ND * NT);
      float ga[2] = {1.f, 1.f};
      if (FMT == LUTQ_NVFP4 && row < a.N) {
#pragma unroll
        for (int w = 0; w < ND; ++w)
          ga[w] = *reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(a.a_rows[w]) +
                                                  int64_t(expert) * a.a_stride + row * 4);
      }
      auto put = [&](int m, float v0, float v1) {
        if (FMT == LUTQ_NVFP4) {
          const float gb = a.b_rows[token0 + m];
          v0 = v0 * ga[0] * gb;
          if (ND == 2) v1 = v1 * ga[1] * gb;
        }
        if (row >= a.N) return;
        const int64_t i = (token0 + m) * a.N + row;
        if (MODE == kMxGateUp) store1<LUTQ_BF16>(a.y, i, silu_mul(v0, v1));
        else store1<LUTQ_FP32>(a.y, i, v0);
      };
      if (split == 1) {
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          if (c >= valid) break;
          uint32_t v[ND][16];
#pragma unroll
          for (int w = 0; w < ND; ++w) tmem_ld_32x32b_x16(d + w * NT + c, v[w]);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < valid)
              put(c + j, __uint_as_float(v[0][j]), __uint_as_float(v[ND - 1][j]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh->acc_empty[b]));
      } else {
        // this block's sums into its own memory, [w][column][row], where the
        // blocks that add up the columns fetch them
        ok = n == 0 || mbar_wait_cluster(smem_addr(&sh->part_empty), uint32_t(n - 1) & 1u, abort,
                                         kMxWaitNs);
        if (!__all_sync(0xffffffffu, ok)) break;
        float* mine = sums + quarter * 32 + lane;
#pragma unroll 1
        for (int c = 0; c < valid; c += 16) {
          uint32_t v[ND][16];
#pragma unroll
          for (int w = 0; w < ND; ++w) tmem_ld_32x32b_x16(d + w * NT + c, v[w]);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
#pragma unroll
            for (int w = 0; w < ND; ++w) mine[(w * NT + c + j) * 128] = __uint_as_float(v[w][j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh->acc_empty[b]));
        if (lane < split) cluster_arrive(cluster_map(smem_addr(&sh->part_full), lane));
        ok = mbar_wait_cluster(smem_addr(&sh->part_full), uint32_t(n) & 1u, abort, kMxWaitNs);
        if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll 1
        for (int j = 0; j < own; ++j) {
          const int col = int(rank) * own + j;
          if (col >= valid) break;
          float part[ND][8], sum[2] = {0.f, 0.f};
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < split) {
#pragma unroll
              for (int w = 0; w < ND; ++w)
                part[w][q] = cluster_ld_f32(
                    cluster_map(smem_addr(mine + (w * NT + col) * 128), uint32_t(q)));
            }
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < split) {
#pragma unroll
              for (int w = 0; w < ND; ++w) sum[w] += part[w][q];
            }
          put(col, sum[0], sum[ND - 1]);
        }
        __syncwarp();
        if (lane < split) cluster_arrive(cluster_map(smem_addr(&sh->part_empty), lane));
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync_all();  // no block leaves while another may fetch from it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::TMEM);
  }
  if (threadIdx.x == 0 && *abort) report(a.dev_status, LUTQ_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ host side

constexpr int kMxSmemMax = 227 * 1024;

template <int FMT, int NT, int MODE>
static cudaError_t launch_one(const CUtensorMap* t, MxGemmArgs a, int64_t tiles, int num_sms,
                              cudaStream_t stream) {
  using Cfg = MxCfg<FMT, NT, MODE>;
  // narrow tiles of one matrix leave room for a second block on the SM; the
  // partial sums of a wide gate-and-up tile would leave none for stages
  constexpr bool two = NT <= 32 && Cfg::ND == 1;
  constexpr int budget = two ? 113 * 1024 : kMxSmemMax;
  const int split =
      mx_split(tiles, a.chunks, two ? 2 : 1, num_sms, Cfg::ND == 2 && NT > 32 ? 1 : 8);
  const int clusters =
      int(std::max<int64_t>(1, std::min(tiles, mx_clusters(split, two ? 2 : 1, num_sms))));
  const int fixed = 1024 + (split > 1 ? Cfg::SUMS : 0) + int(sizeof(MxShared)) +
                    8 * a.experts;
  a.stages = std::min(kMxMaxStages, (budget - fixed) / Cfg::STAGE);
  if (a.stages < 2) return cudaErrorInvalidValue;
  const int smem = std::max(fixed + a.stages * Cfg::STAGE, mx_smem_floor(Cfg::TMEM));
  static bool granted[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  auto kernel = mx_gemm_kernel<FMT, NT, MODE>;
  if (!granted[dev]) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMxSmemMax);
    if (err != cudaSuccess) return err;
    granted[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(clusters * split));
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {unsigned(split), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, t[0], t[1], t[2], t[3], a, split);
}

template <int FMT, int MODE>
static cudaError_t launch_nt(const CUtensorMap* t, const MxGemmArgs& a, int nt, int64_t tiles,
                             int num_sms, cudaStream_t stream) {
  switch (nt) {
    case 16: return launch_one<FMT, 16, MODE>(t, a, tiles, num_sms, stream);
    case 32: return launch_one<FMT, 32, MODE>(t, a, tiles, num_sms, stream);
    case 64: return launch_one<FMT, 64, MODE>(t, a, tiles, num_sms, stream);
    default: return launch_one<FMT, 128, MODE>(t, a, tiles, num_sms, stream);
  }
}

template <int FMT>
static cudaError_t launch_mode(const CUtensorMap* t, const MxGemmArgs& a, int mode, int nt,
                               int64_t tiles, int num_sms, cudaStream_t stream) {
  return mode == kMxGateUp ? launch_nt<FMT, kMxGateUp>(t, a, nt, tiles, num_sms, stream)
                           : launch_nt<FMT, kMxDown>(t, a, nt, tiles, num_sms, stream);
}

cudaError_t launch_mx_gemm(const CUtensorMap* t, const MxGemmArgs& a, int fmt, int mode, int nt,
                           int64_t tiles, int num_sms, cudaStream_t stream) {
  return fmt == LUTQ_MXFP4 ? launch_mode<LUTQ_MXFP4>(t, a, mode, nt, tiles, num_sms, stream)
                           : launch_mode<LUTQ_NVFP4>(t, a, mode, nt, tiles, num_sms, stream);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static EncodeTiledFn enc = nullptr;
  if (enc == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      enc = reinterpret_cast<EncodeTiledFn>(p);
  }
  return enc;
}

static cudaError_t encode(CUtensorMap* map, CUtensorMapDataType type, int dims, const void* base,
                          const cuuint64_t* dim, const cuuint64_t* stride, const cuuint32_t* box,
                          CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return cudaErrorNotSupported;
  const cuuint32_t one[3] = {1, 1, 1};
  CUresult r = enc(map, type, cuuint32_t(dims), const_cast<void*>(base), dim, stride, box, one,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_mx_scale_map(CUtensorMap* map, const void* packed, int64_t rows, int64_t K,
                              int64_t batch, int64_t stride, int fmt) {
  const int per = mx_chunk_bytes(fmt) / 1024;
  const cuuint64_t dims[3] = {
      256, cuuint64_t(mx_ceil(rows, kMxRowTile) * mx_ceil(K, kMxChunk) * per), cuuint64_t(batch)};
  const cuuint64_t strides[2] = {1024, cuuint64_t(stride)};
  const cuuint32_t box[3] = {256, cuuint32_t(per), 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3,
                static_cast<const uint8_t*>(packed) + mx_scale_off(rows, K), dims, strides, box,
                CU_TENSOR_MAP_SWIZZLE_NONE);
}

cudaError_t make_mx_out_map(CUtensorMap* map, void* y, int64_t M, int64_t N, int dtype) {
  const int es = dtype == LUTQ_FP32 ? 4 : 2;
  const cuuint64_t dims[2] = {cuuint64_t(N), cuuint64_t(M)};
  const cuuint64_t strides[1] = {cuuint64_t(N * es)};
  const cuuint32_t box[2] = {32, 32};
  return encode(map, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
                y, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// The codes of `batch` matrices [rows, K/2 bytes], `stride` bytes apart, in
// boxes of 128 bytes x box_rows with the 128-byte swizzle; rows and columns
// beyond a matrix read as zero.
cudaError_t make_mx_map(CUtensorMap* map, const void* codes, int64_t rows, int64_t K,
                        int64_t batch, int64_t stride, int box_rows) {
  const cuuint64_t dims[3] = {cuuint64_t(K / 2), cuuint64_t(rows), cuuint64_t(batch)};
  const cuuint64_t strides[2] = {cuuint64_t(K / 2), cuuint64_t(stride)};
  const cuuint32_t box[3] = {128, cuuint32_t(box_rows), 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, strides, box,
                CU_TENSOR_MAP_SWIZZLE_128B);
}

int mx_tile_tokens(int64_t M) { return M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128; }

// y[M, N] = x w^T.  x: the packed tokens, or (values) M <= 16 rows of values.
cudaError_t launch_mx_product(const void* x, int x_dtype, bool values, int64_t M,
                              const void* packed, int fmt, int64_t N, int64_t K, void* y,
                              int y_dtype, int32_t* dev_status, int num_sms,
                              cudaStream_t stream) {
  const uint8_t* w = static_cast<const uint8_t*>(packed);
  const uint8_t* xp = static_cast<const uint8_t*>(x);
  MxGemmArgs a = {};
  a.y = y;
  a.y_dtype = y_dtype;
  a.dev_status = dev_status;
  a.N = N;
  a.M = M;
  a.K = K;
  if (values) {
    a.x = x;
    a.x_dtype = x_dtype;
    return launch_mx_small(a, packed, nullptr, fmt, kMxPlain, nullptr, 0, 1, num_sms, stream);
  }
  a.a_scales[0] = a.a_scales[1] = w + mx_scale_off(N, K);
  a.a_rows[0] = a.a_rows[1] = reinterpret_cast<const float*>(w + mx_row_off(N, K, fmt));
  a.b_scales = xp + mx_scale_off(M, K);
  a.b_rows = reinterpret_cast<const float*>(xp + mx_row_off(M, K, fmt));
  a.chunks = int(mx_ceil(K, kMxChunk));
  return launch_mx_pair(a, w, nullptr, mx_bytes(N, K, fmt), xp, M, fmt, kMxPlain, 0, num_sms,
                        stream);
}

}  // namespace lutq
