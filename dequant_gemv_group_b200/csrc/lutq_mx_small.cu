// The products of microscaled 4-bit matrices with few tokens, whose values
// are quantized inside the kernel: lutq_mx_gemv (up to 16 tokens), and the
// experts' layer where an expert has a handful of tokens.
//
// Bound by the weights' bytes: the kernel's job is to keep copies of the
// weight tiles in flight from its first microsecond to its last.  A tile is
// 128 weight rows by 16 tokens; a stage holds 256 elements of K of one tile
// (of two matrices for gate and up).  Meanwhile four warps turn the tokens'
// values into codes and scale bytes in shared memory, in the order of the
// tensor core's 128-byte swizzle; they are loaded a round ahead, and stay as
// long as a block's tiles have the same tokens (a block takes neighbouring
// tiles).  A cluster of `split` blocks shares a tile by K, as in
// lutq_mx_gemm.cu; so neither a workspace nor another launch is needed, and
// results do not depend on timing.
//
// Experts: (token, choice) pairs p = t * top_k + j are listed by expert in
// shared memory by every block for itself; a tile takes up to 16 pairs of an
// expert.  Rows of the hidden values and of the outputs are pairs.
//
// Warps: 0 copies, 1 issues, 2..5 read tensor memory and write, 6..9 quantize.
#include <algorithm>
#include <cstring>

#include "lutq_mx_gemm.cuh"
#include "lutq_sm100.cuh"

namespace lutq {

using namespace sm100;

constexpr uint64_t kSmallWaitNs = 2000000000ull;
constexpr int kSmallNT = 16;
constexpr int kSmallStages = 12;
constexpr int kSmallSlots = 64;
constexpr int kSmallThreads = 320;
constexpr int kSmallQuantWarp = 6;
constexpr int kSmallEntry = 4;       // words of an entry of the expert list
constexpr int32_t kNoExpert = 0x7fffffff;
constexpr int kSmallLook = 128;

template <int FMT, int MODE>
struct SmallCfg {
  static constexpr int ND = MODE == kMxGateUp ? 2 : 1;
  static constexpr int CH = mx_chunk_bytes(FMT);
  static constexpr int BLOCKS = CH / 512;
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int STAGE = ND * (A_BYTES + CH);
  static constexpr int B_BYTES = kSmallNT * 128;
  static constexpr int SLOT = B_BYTES + CH;             // a chunk of the tokens
  static constexpr int SUMS = ND * kSmallNT * 128 * 4;  // partial sums of a split tile
  static constexpr int SF_COLS = (ND + 1) * BLOCKS * 4;
  static constexpr int COLS = 2 * ND * kSmallNT + 2 * SF_COLS;
  static constexpr int TMEM = COLS <= 64 ? 64 : COLS <= 128 ? 128 : 256;
  static_assert(COLS <= 256, "");
};

struct alignas(16) SmallShared {
  uint64_t full[kSmallStages], empty[kSmallStages];
  uint64_t bfull[kSmallSlots], bempty[kSmallSlots];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t part_full, part_empty, max_full, drain;
  uint32_t tmem;
  int abort;
  int entries;
  uint32_t row_max[8][kSmallNT];   // the cluster's largest magnitudes per token (nvfp4)
  uint32_t my_max[2][kSmallNT];
  // nvfp4: the tokens' row scales of the last four fills.  A fill is written
  // once the MMAs of the fill before have begun its last tile, so the epilogue
  // is at most two fills behind.
  float row_scale[4][kSmallNT];
};

struct SmallArgs {
  MxGemmArgs g;
  int split;
  int slots;             // chunks of the tokens that shared memory holds
  const int32_t* ids;    // experts: [pairs]
  int pairs, top_k;
};

__device__ __forceinline__ void small_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_ns() - t0 > kSmallWaitNs) return;
}

// Wait for the work before this launch in the stream.
__device__ __forceinline__ void wait_before() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// DT: the type of the values.
template <int FMT, int MODE, int DT>
__global__ void __launch_bounds__(kSmallThreads)
    mx_small_kernel(const __grid_constant__ CUtensorMap tmap_a,
                    const __grid_constant__ CUtensorMap tmap_a2, const SmallArgs p) {
  using Cfg = SmallCfg<FMT, MODE>;
  constexpr int ND = Cfg::ND, CH = Cfg::CH, BLOCKS = Cfg::BLOCKS, NT = kSmallNT;
  const MxGemmArgs& a = p.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int ST = a.stages, split = p.split, slots = p.slots;
  uint8_t* tokens = smem + ST * Cfg::STAGE;
  float* sums = reinterpret_cast<float*>(tokens + slots * Cfg::SLOT);
  SmallShared* sh = reinterpret_cast<SmallShared*>(reinterpret_cast<uint8_t*>(sums) +
                                                   (split > 1 ? Cfg::SUMS : 0));
  // experts: the ids; entries {expert, first place in the list, pairs, -}; the
  // list; what makes the entries
  const int padded = (p.pairs + 3) & ~3;
  int32_t* ids = reinterpret_cast<int32_t*>(sh + 1);
  int32_t* blocks = ids + padded;
  int32_t* entry = blocks + padded;
  int32_t* list = entry + kSmallEntry * padded;
  int32_t* cursor = list + padded;
  const uint32_t sbase = smem_addr(smem);
  // warp-uniform for the compiler, too
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  volatile int* abort = &sh->abort;
  auto full = [&](int s) { return smem_addr(&sh->full[s]); };
  auto empty = [&](int s) { return smem_addr(&sh->empty[s]); };
  auto bfull = [&](int s) { return smem_addr(&sh->bfull[s]); };
  auto bempty = [&](int s) { return smem_addr(&sh->bempty[s]); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < slots; ++s) {
      mbar_init(bfull(s), NT * 8);
      mbar_init(bempty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(&sh->acc_full[b]), 1);
      mbar_init(smem_addr(&sh->acc_empty[b]), 4);
    }
    mbar_init(smem_addr(&sh->part_full), 4 * split);
    mbar_init(smem_addr(&sh->part_empty), 4 * split);
    mbar_init(smem_addr(&sh->max_full), split);
    mbar_init(smem_addr(&sh->drain), 1);
    sh->abort = 0;
    sh->entries = 0;
    mbar_fence_init();
  }
  if (threadIdx.x < 2 * NT) sh->my_max[threadIdx.x / NT][threadIdx.x % NT] = 0u;
  if (warp == 1) {
    tmem_alloc(smem_addr(&sh->tmem), Cfg::TMEM);
    tmem_relinquish();
  }
  // The down product follows straight after the gate and up product of the same
  // call, which waited for all work before it and only then let this launch
  // start: the ids and the weights are there, and only the hidden values must
  // be waited for.
  if (MODE != kMxDown) wait_before();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t rank = split > 1 ? cluster_ctarank() : 0u;
  const int cluster = blockIdx.x / split, clusters = gridDim.x / split;
  const int c0 = int(int64_t(a.chunks) * rank / split);
  const int nch = int(int64_t(a.chunks) * (rank + 1) / split) - c0;
  auto load_stage = [&](int s, int expert, int mt, int c) {
    const int64_t off = int64_t(expert) * a.a_stride + (int64_t(mt) * a.chunks + c0 + c) * CH;
    const uint32_t st = sbase + s * Cfg::STAGE, sf = st + ND * Cfg::A_BYTES;
    mbar_expect_tx(full(s), Cfg::STAGE);
    tma_3d_g2s(st, &tmap_a, (c0 + c) * 128, mt * 128, expert, full(s));
    if (ND == 2) tma_3d_g2s(st + Cfg::A_BYTES, &tmap_a2, (c0 + c) * 128, mt * 128, expert, full(s));
    bulk_g2s(sf, a.a_scales[0] + off, CH, full(s));
    if (ND == 2) bulk_g2s(sf + CH, a.a_scales[1] + off, CH, full(s));
  };
  if (MODE != kMxPlain) {
#pragma unroll 1
    for (int i = threadIdx.x; i < padded; i += kSmallThreads) {
      const int id = i < p.pairs ? p.ids[i] : -1;
      ids[i] = uint32_t(id) < uint32_t(a.experts) ? id : kNoExpert;
      if (i >= p.pairs) blocks[i] = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_arrive_all();  // this block's barriers are set up
  if (MODE != kMxPlain) {
    // The list of pairs by expert, in their order (the same in all blocks of a
    // cluster).  Every block makes it before its first copy, so it is made in
    // the quicker of two ways: few pairs, a thread finds its pair's place by
    // looking at all others (8 pairs: 2 us quicker than the other way; 148: the
    // same; 256: 2 us slower); more, counts by expert, a scan, and placing by
    // warp matches.
    if (p.pairs <= kSmallLook) {
      auto look = [&](const int32_t* of, auto&& each) {
#pragma unroll 1
        for (int q = 0; q < padded; q += 4) {
          const int4 d = *reinterpret_cast<const int4*>(of + q);
          each(q, d.x);
          each(q + 1, d.y);
          each(q + 2, d.z);
          each(q + 3, d.w);
        }
      };
#pragma unroll 1
      for (int i = threadIdx.x; i < p.pairs; i += kSmallThreads) {
        const int id = ids[i];
        int place = 0, before = 0, count = 0;
        look(ids, [&](int q, int o) {
          place += uint32_t(o) < uint32_t(id);
          count += o == id;
          before += o == id && q < i;
        });
        if (id == kNoExpert) {
          blocks[i] = 0;
          continue;
        }
        list[place + before] = i;
        // the first pair of each 16 of an expert makes an entry, below
        blocks[i] = before == 0 ? (count + NT - 1) / NT : 0;
        if (before % NT == 0) {
          const int left = count - before;
          cursor[i] = ((place + before) << 8) | (left < NT ? left : NT);
        }
      }
      __syncthreads();
#pragma unroll 1
      for (int i = threadIdx.x; i < p.pairs; i += kSmallThreads) {
        const int id = ids[i];
        int at = 0, before = 0, all = 0;
#pragma unroll 1
        for (int q = 0; q < padded; q += 4) {
          const int4 o = *reinterpret_cast<const int4*>(ids + q);
          const int4 n = *reinterpret_cast<const int4*>(blocks + q);
          at += (uint32_t(o.x) < uint32_t(id) ? n.x : 0) +
                (uint32_t(o.y) < uint32_t(id) ? n.y : 0) +
                (uint32_t(o.z) < uint32_t(id) ? n.z : 0) + (uint32_t(o.w) < uint32_t(id) ? n.w : 0);
          all += n.x + n.y + n.z + n.w;
          before += (o.x == id && q < i) + (o.y == id && q + 1 < i) + (o.z == id && q + 2 < i) +
                    (o.w == id && q + 3 < i);
        }
        if (i == 0) sh->entries = all;
        if (id == kNoExpert || before % NT != 0) continue;
        int32_t* en = entry + kSmallEntry * (at + before / NT);
        en[0] = id;
        en[1] = cursor[i] >> 8;
        en[2] = cursor[i] & 255;
      }
      __syncthreads();
    } else {
#pragma unroll 1
      for (int e = threadIdx.x; e < a.experts; e += kSmallThreads) cursor[e] = 0;
      __syncthreads();
#pragma unroll 1
      for (int i = threadIdx.x; i < p.pairs; i += kSmallThreads)
        if (ids[i] != kNoExpert) atomicAdd(&cursor[ids[i]], 1);
      __syncthreads();
      if (warp == 0) {
        // entries of the experts in use, and where their pairs begin
        int place = 0, n = 0;
#pragma unroll 1
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
          const int e = e0 + lane, c = e < a.experts ? cursor[e] : 0, k = (c + NT - 1) / NT;
          int both = c | (k << 16);  // inclusive sums over the lanes
#pragma unroll
          for (int x = 1; x < 32; x *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, both, x);
            if (lane >= x) both += v;
          }
          const int pc = both & 0xffff, pk = both >> 16;
#pragma unroll 1
          for (int i = 0; i < k; ++i) {
            int32_t* en = entry + kSmallEntry * (n + pk - k + i);
            en[0] = e;
            en[1] = place + pc - c + i * NT;
            en[2] = min(NT, c - i * NT);
          }
          if (e < a.experts) cursor[e] = place + pc - c;
          both = __shfl_sync(0xffffffffu, both, 31);
          place += both & 0xffff;
          n += both >> 16;
        }
        if (lane == 0) sh->entries = n;
        __syncwarp();
#pragma unroll 1
        for (int i0 = 0; i0 < p.pairs; i0 += 32) {
          const int i = i0 + lane, id = i < p.pairs ? ids[i] : kNoExpert;
          const uint32_t same = __match_any_sync(0xffffffffu, id);
          const int at = id != kNoExpert ? cursor[id] : 0;
          const int before = __popc(same & ((1u << lane) - 1u));
          __syncwarp();
          if (id != kNoExpert) {
            list[at + before] = i;
            if (before == 0) cursor[id] = at + __popc(same);
          }
          __syncwarp();
        }
      }
      __syncthreads();
    }
  }
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh->tmem, 0);
  const int ntiles = (MODE == kMxPlain ? 1 : sh->entries) * a.mtiles;
  const int t0 = int(int64_t(ntiles) * cluster / clusters);
  const int t1 = int(int64_t(ntiles) * (cluster + 1) / clusters);
  // Tokens in shared memory: all chunks of a tile's, kept for the tiles of the
  // same tokens that follow (a fill), or a ring, filled for every tile.
  const bool keep = nch <= slots;
  auto entry_of = [&](int t) { return MODE == kMxPlain ? 0 : t / a.mtiles; };
  auto opens = [&](int t) { return !keep || t == t0 || entry_of(t) != entry_of(t - 1); };
  auto closes = [&](int t) { return !keep || t + 1 == t1 || entry_of(t) != entry_of(t + 1); };
  const bool once = MODE == kMxPlain && keep;
  struct Tile {
    int expert, mt, at, valid;
  };
  auto tile = [&](int t) {
    Tile r{0, t, 0, int(a.M)};
    if (MODE != kMxPlain) {
      const int32_t* en = entry + kSmallEntry * (t / a.mtiles);
      r = Tile{en[0], t % a.mtiles, en[1], en[2]};
    }
    return r;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ weights
    int s = 0;
    uint32_t ph = 1;
    int issued = 0;
    bool ok = true;
    for (int t = t0; ok && t < t1; ++t) {
      const Tile r = tile(t);
      for (int c = 0; c < nch; ++c) {
        ok = mbar_wait(empty(s), ph, abort, kSmallWaitNs);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        if (elect_one()) load_stage(s, r.expert, r.mt, c);
        __syncwarp();
        ++issued;
        if (++s == ST) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // given up: the copies in flight must land before the block may exit
    if (__any_sync(0xffffffffu, *abort))
      for (int i = max(0, issued - ST); i < issued; ++i)
        small_drain(full(i % ST), uint32_t(i / ST) & 1u);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    constexpr bool E8 = FMT == LUTQ_MXFP4;
    constexpr uint32_t idesc = idesc_e2m1(128, NT, E8, 0), id2 = idesc_e2m1(0, 0, false, 2);
    int s = 0, it = 0, n = 0, b = 0;
    uint32_t ph = 0, bph = keep ? 1 : 0;
    bool ok = true, any = false;
    for (int t = t0; ok && t < t1; ++t, ++n) {
      const int acc = n & 1;
      ok = mbar_wait(smem_addr(&sh->acc_empty[acc]), (uint32_t(n >> 1) & 1u) ^ 1u, abort,
                     kSmallWaitNs);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const uint32_t d = tmem + uint32_t(acc * ND * NT);
      if (keep) {
        b = 0;
        if (opens(t)) bph ^= 1;
      }
      const bool release = closes(t);
      for (int c = 0; c < nch; ++c, ++it) {
        ok = mbar_wait(bfull(b), bph, abort, kSmallWaitNs) &&
             mbar_wait(full(s), ph, abort, kSmallWaitNs);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        tc_fence_after();
        const uint32_t st = desc_lo(sbase + s * Cfg::STAGE);
        const uint32_t sf = st + ((ND * Cfg::A_BYTES) >> 4);
        const uint32_t bl = desc_lo(smem_addr(tokens) + b * Cfg::SLOT);
        const uint32_t bsf = bl + (Cfg::B_BYTES >> 4);
        const uint32_t sf_tmem = tmem + uint32_t(2 * ND * NT + (it & 1) * Cfg::SF_COLS);
        const uint32_t sb_tmem = sf_tmem + 4 * ND * BLOCKS;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < ND * BLOCKS; ++i) tmem_cp_scales(sf_tmem + 4 * i, sf + 32 * i);
#pragma unroll
          for (int i = 0; i < BLOCKS; ++i) tmem_cp_scales(sb_tmem + 4 * i, bsf + 32 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // mxfp4: a block holds the scales of two MMAs, nvfp4: of one
            const int blk = E8 ? j >> 1 : j;
#pragma unroll
            for (int w = 0; w < ND; ++w)
              mma_e2m1_ss<!E8>(d + w * NT, st + ((w * Cfg::A_BYTES) >> 4) + 2 * j, bl + 2 * j,
                               E8 && (j & 1) ? idesc | id2 : idesc,
                               sf_tmem + 4 * (w * BLOCKS + blk), sb_tmem + 4 * blk,
                               (c > 0 || j > 0) ? 1u : 0u);
          }
          mma_commit(empty(s));
          if (release) mma_commit(bempty(b));
        }
        __syncwarp();
        any = true;
        if (++s == ST) {
          s = 0;
          ph ^= 1;
        }
        if (++b == slots && !keep) {
          b = 0;
          bph ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) mma_commit(smem_addr(&sh->acc_full[acc]));
      __syncwarp();
    }
    if (__any_sync(0xffffffffu, *abort) && any) {
      if (elect_one()) mma_commit(smem_addr(&sh->drain));
      __syncwarp();
      small_drain(smem_addr(&sh->drain), 0);
    }
  } else {
    bool met = split == 1;  // the other blocks' barriers are known to be set up
    // Values into codes, by warps 6..9; where that is done once, by the
    // epilogue's warps as well, which have nothing else to do yet.
    if (warp >= kSmallQuantWarp || once) {
      if (MODE == kMxDown) wait_before();  // the hidden values
      const int th = int(threadIdx.x) - (once ? 64 : kSmallQuantWarp * 32);
      const int nq = once ? 256 : 128;
      constexpr int64_t esize = DT == LUTQ_FP32 ? 4 : 2;
      const uint8_t* x = static_cast<const uint8_t*>(a.x);
      bool ok = true, bad = false;
      float g = 1.f, g_inv = 1.f;
      int ring = 0;   // chunks quantized so far (slot and phase of the next)
      int fill = -1;  // fills
      for (int t = t0; t < t1; ++t) {
        if (!opens(t)) continue;
        ++fill;
        // (the warps share barriers: they go on together or not at all)
        if (!group_all(1, nq, ok)) break;
        const Tile r = tile(t);
        // 8 threads take a token's chunk (a block of 32 elements each); as many
        // chunks at a time as the tokens leave threads for
        int rows = 1;
        while (rows < r.valid) rows *= 2;
        // (no more than there are slots: a warp's threads wait for their slots
        // together, so none may need another's chunk of the same round)
        int per = nq / (8 * rows);
        while (per > slots) per /= 2;
        const int q = th & 7, i = (th >> 3) & (rows - 1), lead = (th >> 3) / rows;
        const bool live = i < r.valid;
        int64_t src = 0;
        if (live) {
          src = i;
          if (MODE == kMxGateUp) src = list[r.at + i] / p.top_k;
          if (MODE == kMxDown) src = list[r.at + i];
        }
        const uint8_t* xr = x + src * a.K * esize;
        auto load32 = [&](int c, Raw8<DT> (&raw)[4]) {
          const int64_t k = int64_t(c) * kMxChunk + q * 32;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            raw[j] = Raw8<DT>{};
            if (live && k < a.K) raw[j] = load_raw8<DT>(xr, k + 8 * j);
          }
        };
        if (FMT == LUTQ_NVFP4 && (MODE != kMxPlain || fill == 0)) {
          // the token's largest finite magnitude.  Plain: of this block's
          // chunks, then the cluster's; experts: of the whole row
          const int m0 = MODE == kMxPlain ? c0 : 0, m1 = MODE == kMxPlain ? c0 + nch : a.chunks;
          const int pc = MODE == kMxPlain ? 0 : fill & 1;
          uint32_t m = 0;
#pragma unroll 2
          for (int c = lead < per ? m0 + lead : m1; c < m1; c += per) {
            Raw8<DT> raw[4];
            load32(c, raw);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t b = max_raw8<DT>(raw[j]);
              m = max(m, b < raw_inf<DT>() ? max_bits_f32<DT>(b) : finite_max8<DT>(raw[j]));
            }
          }
          if (live && lead < per) atomicMax(&sh->my_max[pc][i], m);
          asm volatile("bar.sync 1, %0;" ::"r"(nq) : "memory");
          if (MODE == kMxPlain && split > 1) {
            cluster_wait_all();
            met = true;
            if (th < NT)
              for (int k = 0; k < split; ++k)
                cluster_st_u32(cluster_map(smem_addr(&sh->row_max[rank][th]), k),
                               sh->my_max[0][th]);
            __syncwarp();
            if (th < split) cluster_arrive(cluster_map(smem_addr(&sh->max_full), th));
            ok = mbar_wait_cluster(smem_addr(&sh->max_full), 0, abort, kSmallWaitNs);
            if (!(ok = group_all(1, nq, ok))) break;
            m = 0;
            for (int k = 0; k < split; ++k) m = max(m, sh->row_max[k][i]);
          } else {
            m = sh->my_max[pc][i];
          }
          g = nv_row_scale(m);
          g_inv = nv_row_scale_inverse(g);
          if (MODE != kMxPlain) {
            asm volatile("bar.sync 1, %0;" ::"r"(nq) : "memory");  // all have read my_max
            if (th < NT) sh->my_max[pc][th] = 0u;
          }
        }
        Raw8<DT> raw[4];
        if (lead < per && lead < nch) load32(c0 + lead, raw);
        for (int c = lead < per ? lead : nch; c < nch; c += per) {
          const int f = keep ? fill * slots + c : ring + c, slot = f % slots;
          uint32_t sc[2] = {0u, 0u}, codes[4] = {0u, 0u, 0u, 0u};
          constexpr int H = FMT == LUTQ_MXFP4 ? 1 : 2;  // blocks per 32 elements
          if (live) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
              uint32_t m = 0;
#pragma unroll
              for (int w = 0; w < 4 / H; ++w) m = max(m, max_raw8<DT>(raw[h * 2 + w]));
              if (m >= raw_inf<DT>()) {
                bad = true;
                sc[h] = FMT == LUTQ_MXFP4 ? 0xFFu : 0x7Fu;
              } else {
                m = max_bits_f32<DT>(m);
                sc[h] = FMT == LUTQ_MXFP4 ? e8m0_byte(m) : nv_scale_byte<DT>(m, g_inv);
#pragma unroll
                for (int w = 0; w < 4 / H; ++w) {
                  float v[8];
                  widen8<DT>(raw[h * 2 + w], v);
                  codes[h * 2 + w] = mx_codes8<FMT, DT>(v, sc[h], g, g_inv);
                }
              }
            }
            if (int64_t(c0 + c) * kMxChunk + q * 32 >= a.K) sc[0] = sc[1] = 0u;
          }
          if (c + per < nch) load32(c0 + c + per, raw);  // a round ahead
          ok = mbar_wait(bempty(slot), (uint32_t(f / slots) & 1u) ^ 1u, abort, kSmallWaitNs);
          if (!ok) break;
          if (FMT == LUTQ_NVFP4 && c == 0 && q == 0 && live) sh->row_scale[fill & 3][i] = g;
          uint8_t* bp = tokens + slot * Cfg::SLOT;
          if (live) {
            *reinterpret_cast<uint4*>(bp + i * 128 + ((q ^ (i & 7)) * 16)) =
                make_uint4(codes[0], codes[1], codes[2], codes[3]);
            uint8_t* sf = bp + Cfg::B_BYTES + i * 16;
            if (FMT == LUTQ_MXFP4)
              sf[(q >> 2) * 512 + (q & 3)] = uint8_t(sc[0]);
            else
              *reinterpret_cast<uint16_t*>(sf + (q >> 1) * 512 + (q & 1) * 2) =
                  uint16_t(sc[0] | (sc[1] << 8));
          }
          fence_async_shared();
          // 8 * rows threads have this chunk; the barrier counts 128 arrivals
          mbar_arrive_n(bfull(slot), uint32_t(NT / rows));
        }
        ring += nch;
      }
      if (bad) report(a.dev_status, LUTQ_ERR_NONFINITE);
    }
    if (!met) cluster_wait_all();
    if (warp < kSmallQuantWarp) {
      const int quarter = warp & 3;
      int n = 0, fill = -1;
      bool ok = true;
      const int own = NT / split;  // columns of a split tile that this block sums
      for (int t = t0; ok && t < t1; ++t, ++n) {
        const Tile r = tile(t);
        if (opens(t)) ++fill;
        const int acc = n & 1;
        const int64_t row = int64_t(r.mt) * 128 + quarter * 32 + lane;
        float ga[2] = {1.f, 1.f};
        if (FMT == LUTQ_NVFP4 && row < a.N) {
#pragma unroll
          for (int w = 0; w < ND; ++w)
            ga[w] = *reinterpret_cast<const float*>(reinterpret_cast<const uint8_t*>(a.a_rows[w]) +
                                                    int64_t(r.expert) * a.a_stride + row * 4);
        }
        ok = mbar_wait(smem_addr(&sh->acc_full[acc]), uint32_t(n >> 1) & 1u, abort, kSmallWaitNs);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        auto put = [&](int m, float v0, float v1) {
          if (FMT == LUTQ_NVFP4) {
            const float gb = sh->row_scale[fill & 3][m];
            v0 = v0 * ga[0] * gb;
            if (ND == 2) v1 = v1 * ga[1] * gb;
          }
          if (row >= a.N) return;
          const int64_t at = int64_t(MODE == kMxPlain ? m : list[r.at + m]) * a.N + row;
          if (MODE == kMxGateUp) store1<LUTQ_BF16>(a.y, at, silu_mul(v0, v1));
          else if (MODE == kMxDown) store1<LUTQ_FP32>(a.y, at, v0);
          else if (a.y_dtype == LUTQ_FP32) store1<LUTQ_FP32>(a.y, at, v0);
          else if (a.y_dtype == LUTQ_BF16) store1<LUTQ_BF16>(a.y, at, v0);
          else store1<LUTQ_FP16>(a.y, at, v0);
        };
        const uint32_t d = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(acc * ND * NT);
        uint32_t v[ND][16];
#pragma unroll
        for (int w = 0; w < ND; ++w) tmem_ld_32x32b_x16(d + w * NT, v[w]);
        tmem_wait_ld();
        if (split == 1) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
            if (j < r.valid) put(j, __uint_as_float(v[0][j]), __uint_as_float(v[ND - 1][j]));
          // (behind the reads of row_scale: see there)
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh->acc_empty[acc]));
        } else {
          // this block's sums into its own memory, [w][column][row], where the
          // blocks that add up the columns fetch them
          ok = n == 0 || mbar_wait_cluster(smem_addr(&sh->part_empty), uint32_t(n - 1) & 1u, abort,
                                           kSmallWaitNs);
          if (!__all_sync(0xffffffffu, ok)) break;
          float* mine = sums + quarter * 32 + lane;
#pragma unroll
          for (int j = 0; j < NT; ++j)
            if (j < r.valid) {
#pragma unroll
              for (int w = 0; w < ND; ++w) mine[(w * NT + j) * 128] = __uint_as_float(v[w][j]);
            }
          __syncwarp();
          if (lane < split) cluster_arrive(cluster_map(smem_addr(&sh->part_full), lane));
          ok = mbar_wait_cluster(smem_addr(&sh->part_full), uint32_t(n) & 1u, abort, kSmallWaitNs);
          if (!__all_sync(0xffffffffu, ok)) break;
          for (int j = 0; j < own; ++j) {
            const int col = int(rank) * own + j;
            if (col >= r.valid) break;
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
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh->acc_empty[acc]));
        }
      }
    }
  }

  __syncwarp();
  if (split > 1 && warp < 2) cluster_wait_all();  // (the other warps have)
  if (MODE == kMxDown) wait_before();  // no thread is done before the work it follows
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

// A launch's shape: blocks that share a tile by K, blocks on a multiprocessor,
// and what follows from them.
struct SmallShape {
  int split, per_sm, clusters, slots, stages, smem;
  bool ok;
};

template <int FMT, int MODE>
static SmallShape small_shape(const SmallArgs& p, int64_t tiles, int split, int per_sm,
                              int num_sms) {
  using Cfg = SmallCfg<FMT, MODE>;
  const int budget = (per_sm == 2 ? 113 : 227) * 1024;
  SmallShape s = {split, per_sm};
  s.clusters = int(std::max<int64_t>(1, std::min(tiles, mx_clusters(split, per_sm, num_sms))));
  const int fixed = 1024 + (split > 1 ? Cfg::SUMS : 0) + int(sizeof(SmallShared)) +
                    (MODE != kMxPlain
                         ? 4 * ((kSmallEntry + 4) * ((p.pairs + 3) & ~3) + p.g.experts)
                         : 0);
  // the tokens' chunks, as far as four stages of weights leave room
  s.slots = std::min({int(mx_ceil(p.g.chunks, split)), kSmallSlots,
                      (budget - fixed - 4 * Cfg::STAGE) / Cfg::SLOT});
  s.stages = std::min(kSmallStages, (budget - fixed - s.slots * Cfg::SLOT) / Cfg::STAGE);
  s.smem = std::max(fixed + s.slots * Cfg::SLOT + s.stages * Cfg::STAGE, mx_smem_floor(Cfg::TMEM));
  s.ok = s.slots >= 1 && (split == 1 || split <= p.g.chunks);
  return s;
}

// What a plain product of a shape takes beyond what all of them do, in us: the terms
// fitted to 1024 x 4096 .. 28672 x 8192 and 8192 x 28672 in both formats at 1,
// 6 and 16 tokens.  Of the eight shapes it takes one that is 2 % slower than
// the best on average and 13 % at worst; as many splits as fill two blocks a
// multiprocessor, the rule before, was 15 % slower on average.
template <int FMT>
static float small_cost(const SmallArgs& p, int64_t tiles, const SmallShape& s, int num_sms) {
  using Cfg = SmallCfg<FMT, kMxPlain>;
  const int per = s.clusters * s.split > num_sms ? s.per_sm : 1;  // blocks where they are most
  const float rounds = float(mx_ceil(tiles, s.clusters));
  const int chunks = int(mx_ceil(p.g.chunks, s.split));  // of a block in a tile
  int rows = 1;
  while (rows < p.g.M) rows *= 2;
  // quantizing: 13 ns a token's chunk, again for every tile if they do not all fit
  const float quantize = .013f * rows * chunks * per * (chunks <= s.slots ? 1.f : rounds);
  // weights: 8 TB/s in all, 72 GB/s a multiprocessor, a stage at 1.2 us
  const float stage = Cfg::STAGE / 1024.f;
  const float weights = std::max(
      float(tiles) * p.g.chunks * stage / 8000.f,
      rounds * chunks * std::max(per * stage / 72.f, 1.2f / s.stages));
  // adding up; all of shared memory: no start beside the launch before
  const float rest = (s.split > 1 ? .9f + 1.6f * rounds : .35f * rounds) +
                     (s.per_sm == 1 ? .6f : 0.f) + .15f * (per - 1);
  return quantize + weights + rest;
}

template <int FMT, int MODE, int DT>
static cudaError_t launch_one(const CUtensorMap* t, SmallArgs p, int64_t tiles, int num_sms,
                              cudaStream_t stream) {
  using Cfg = SmallCfg<FMT, MODE>;
  static_assert(Cfg::TMEM <= 256, "");
  SmallShape best = {};
  if constexpr (MODE == kMxPlain) {
    float least = 0.f;
    for (int per_sm = 1; per_sm <= 2; ++per_sm)
      for (int split = 1; split <= 8; split *= 2) {
        const SmallShape s = small_shape<FMT, MODE>(p, tiles, split, per_sm, num_sms);
        if (!s.ok) continue;
        const float cost = small_cost<FMT>(p, tiles, s, num_sms);
        if (best.ok && cost >= least) continue;
        best = s;
        least = cost;
      }
  } else {
    // two blocks on a multiprocessor where a stage is one matrix
    constexpr int per_sm = Cfg::ND == 1 ? 2 : 1;
    best = small_shape<FMT, MODE>(p, tiles, mx_split(tiles, p.g.chunks, per_sm, num_sms, 8), per_sm,
                                  num_sms);
  }
  if (!best.ok) return cudaErrorInvalidValue;
  p.split = best.split;
  p.slots = best.slots;
  p.g.stages = best.stages;
  auto kernel = mx_small_kernel<FMT, MODE, DT>;
  static bool granted[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!granted[dev]) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (err != cudaSuccess) return err;
    granted[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(best.clusters * p.split));
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = size_t(best.smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {unsigned(p.split), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, t[0], t[1], p);
}

template <int FMT, int MODE>
static cudaError_t launch_dtype(const CUtensorMap* t, const SmallArgs& p, int64_t tiles,
                                int num_sms, cudaStream_t stream) {
  if (MODE == kMxDown || p.g.x_dtype == LUTQ_BF16)
    return launch_one<FMT, MODE, LUTQ_BF16>(t, p, tiles, num_sms, stream);
  if constexpr (MODE != kMxDown) {
    if (p.g.x_dtype == LUTQ_FP16)
      return launch_one<FMT, MODE, LUTQ_FP16>(t, p, tiles, num_sms, stream);
    return launch_one<FMT, MODE, LUTQ_FP32>(t, p, tiles, num_sms, stream);
  }
  return cudaErrorInvalidValue;
}

template <int FMT>
static cudaError_t launch_mode(const CUtensorMap* t, const SmallArgs& p, int mode, int64_t tiles,
                               int num_sms, cudaStream_t stream) {
  if (mode == kMxGateUp) return launch_dtype<FMT, kMxGateUp>(t, p, tiles, num_sms, stream);
  if (mode == kMxDown) return launch_dtype<FMT, kMxDown>(t, p, tiles, num_sms, stream);
  return launch_dtype<FMT, kMxPlain>(t, p, tiles, num_sms, stream);
}

// Pairs whose experts' list fits a block's shared memory beside the stages.
bool mx_small_fits(int64_t pairs, int experts) { return pairs <= 512 && experts <= 1024; }

cudaError_t launch_mx_small(MxGemmArgs g, const void* weights, const void* weights2, int fmt,
                            int mode, const int32_t* ids, int pairs, int top_k, int num_sms,
                            cudaStream_t stream) {
  CUtensorMap t[2];
  std::memset(t, 0, sizeof(t));
  const int64_t bytes = mx_bytes(g.N, g.K, fmt);
  const int64_t batch = std::max(1, g.experts);
  const void* w[2] = {weights, weights2 != nullptr ? weights2 : weights};
  for (int i = 0; i < (mode == kMxGateUp ? 2 : 1); ++i) {
    const uint8_t* b = static_cast<const uint8_t*>(w[i]);
    const cudaError_t err = make_mx_map(&t[i], b, g.N, g.K, batch, bytes, 128);
    if (err != cudaSuccess) return err;
    g.a_scales[i] = b + mx_scale_off(g.N, g.K);
    g.a_rows[i] = reinterpret_cast<const float*>(b + mx_row_off(g.N, g.K, fmt));
  }
  g.a_stride = bytes;
  g.chunks = int(mx_ceil(g.K, kMxChunk));
  g.mtiles = int(mx_ceil(g.N, 128));
  SmallArgs p = {};
  p.g = g;
  p.ids = ids;
  p.pairs = pairs;
  p.top_k = top_k;
  const int64_t tiles = int64_t(g.mtiles) * (mode == kMxPlain ? 1 : std::min(g.experts, pairs));
  return fmt == LUTQ_MXFP4 ? launch_mode<LUTQ_MXFP4>(t, p, mode, tiles, num_sms, stream)
                           : launch_mode<LUTQ_NVFP4>(t, p, mode, tiles, num_sms, stream);
}

}  // namespace lutq
