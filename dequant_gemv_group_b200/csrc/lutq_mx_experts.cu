// A mixture-of-experts feed-forward layer on microscaled 4-bit weights:
//   y[t] = sum_j weights[t, j] * W_down_e (silu(W_gate_e x[t]) * (W_up_e x[t])),
//   e = ids[t, j],
// with x and the hidden values quantized like the weights, so that both
// products run on the tensor cores as they are (lutq_mx_gemm.cu).
//
// (token, choice) pairs are laid out by expert: expert e's rows begin at a
// multiple of 128 (the height of a scale block) and keep the order of the
// pairs.  So does every tile of up to nt rows (fewer than 128 for small
// batches: an expert has more rows than one tile only where tokens name it
// more than once).  Steps: plan (rows of every expert), x quantized into its rows, gate
// and up product with silu, hidden values quantized (by that product for many
// tokens in mxfp4, else a launch), down product, weighted sum over a token's
// choices in their order.  Where an expert has a handful of
// pairs: gate and up, down, sum, with the tokens quantized inside.  Rows do
// not depend on one another.
#include <algorithm>
#include <cstring>

#include "lutq_mx_gemm.cuh"

namespace lutq {

constexpr int kPlanThreads = 512;
// Pairs an expert, at most, for the kernel of few tokens; beyond, tokens are
// packed first (six launches).  Measured, kernel of few tokens / packed, us, by
// pairs an expert:
//   mxfp4: 8 experts of 4096 x 2048: 6 33.4 / 35.7, 8 36.6 / 35.9, 12 43.2 /
//     38.2; 64 of 4096 x 2048: 4 148 / 154, 8 158 / 158; 60 of 2048 x 1440: 6
//     67.4 / 69.9, 8 73.2 / 71.8;
//   nvfp4 (a row's maximum first): 64 of 4096 x 2048: 2.5 145 / 154, 3 187 /
//     159, 4 171 / 163; 60 of 2048 x 1440: 3 65.9 / 71.9, 4 74.3 / 72.9, 8 99 /
//     83; 8 of 4096 x 2048: 3 33.9 / 38.6, 4 36.4 / 39.5, 6 49.5 / 40.4.
constexpr int64_t kSmallPairsMx = 8, kSmallPairsNv = 3;

// More pairs an expert: block pairs (lutq_mx_pair.cu).  Measured, block pairs /
// lutq_mx_gemm.cu, us, by pairs an expert:
//   mxfp4: 8 experts of 4096 x 2048: 16 40.5 / 39.3, 24 41.4 / 41.4, 30 42.5 /
//     42.8; 60 of 2048 x 1440: 16 86.6 / 77.9, 27 87.5 / 84.3; 64 of 4096 x
//     1024: 25 116 / 111;
//   nvfp4: 47.2 / 45.3, 47.5 / 47.4, 48.7 / 49.8; 105 / 96, 107.8 / 107.7;
//     132 / 137.
constexpr int64_t kWidePairs = 24;

// The plan of a call (int32 arrays in the workspace).
struct MoePlan {
  int32_t* counts;  // [E] pairs of an expert
  int32_t* bases;   // [E] its first row
  int32_t* slot;    // [pairs] a pair's row, or -1 (id outside 0..E-1)
  int nt_log2;      // pairs of a tile, a power of two up to 128
};
// The place of an expert's i-th pair behind its first row, and the rows of n
// pairs: tiles begin at multiples of 128 rows.
__device__ __forceinline__ int moe_place(const MoePlan& p, int i) {
  return (i >> p.nt_log2) * 128 + (i & ((1 << p.nt_log2) - 1));
}
__device__ __forceinline__ int moe_height(const MoePlan& p, int n) {
  return ((n + (1 << p.nt_log2) - 1) >> p.nt_log2) * 128;
}

// Four ids from place i on, -1 behind the end.
__device__ __forceinline__ int4 load_ids(const int32_t* ids, int i, int end, bool aligned) {
  if (aligned && i + 4 <= end) return *reinterpret_cast<const int4*>(ids + i);
  return make_int4(i < end ? ids[i] : -1, i + 1 < end ? ids[i + 1] : -1,
                   i + 2 < end ? ids[i + 2] : -1, i + 3 < end ? ids[i + 3] : -1);
}

// A block for each expert e adds up the rows before its own from all experts'
// counts and hands its rows out: each warp owns a run of pairs, 128 at a time,
// and a scan over the warps' and the lanes' counts keeps the pairs' order.
// PLAN_ALL: every block counts all experts' pairs itself; many pairs: a launch
// before (PLAN_COUNT) counts them, each block its expert's.  A layer with one
// launch / two: 1600 pairs 88.9 / 89.1 us, 8192 181.8 / 181.5 and 127.5 / 127.9
// (64 and 256 experts), 16384 294 / 291, 32768 498 / 488.
enum { PLAN_COUNT, PLAN_PLACE, PLAN_ALL };
constexpr int kPlanAll = 1 << 13;
template <int STEP>
__global__ void __launch_bounds__(kPlanThreads)
    moe_plan_kernel(const int32_t* __restrict__ ids, int pairs, int E, MoePlan p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int W = kPlanThreads / 32;
  constexpr bool ALL = STEP == PLAN_ALL;
  __shared__ int32_t warp_count[W];
  __shared__ int32_t base_s;
  __shared__ int32_t of[ALL ? 1024 : 1];  // pairs of every expert
  const int e = blockIdx.x, th = threadIdx.x, lane = th & 31, warp = th >> 5;
  const bool aligned = (reinterpret_cast<uintptr_t>(ids) & 15u) == 0;
  if (th == 0) base_s = 0;
  if (ALL) {
    for (int i = th; i < E; i += kPlanThreads) of[i] = 0;
    __syncthreads();
  }
  const int run = (pairs + W * 128 - 1) / (W * 128) * 128;
  const int i0 = min(pairs, warp * run), i1 = min(pairs, i0 + run);
  int mine = 0;
#pragma unroll 4
  for (int i = i0 + 4 * lane; i < i1; i += 128) {
    const int4 d = load_ids(ids, i, i1, aligned);
    mine += (d.x == e) + (d.y == e) + (d.z == e) + (d.w == e);
    if (ALL) {
      if (uint32_t(d.x) < uint32_t(e)) atomicAdd(&of[d.x], 1);
      if (uint32_t(d.y) < uint32_t(e)) atomicAdd(&of[d.y], 1);
      if (uint32_t(d.z) < uint32_t(e)) atomicAdd(&of[d.z], 1);
      if (uint32_t(d.w) < uint32_t(e)) atomicAdd(&of[d.w], 1);
    }
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) warp_count[warp] = mine;
  __syncthreads();
  if (STEP != PLAN_PLACE && warp == 0) {
    const int c = __reduce_add_sync(0xffffffffu, lane < W ? warp_count[lane] : 0);
    if (lane == 0) p.counts[e] = c;
  }
  if (STEP == PLAN_COUNT) return;
  int before = 0;
  for (int i = th; i < e; i += kPlanThreads)
    before += moe_height(p, ALL ? of[i] : p.counts[i]);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) atomicAdd(&base_s, before);
  __syncthreads();
  const int base = base_s;
  if (th == 0) p.bases[e] = base;
  if (e == 0) {  // pairs of no expert
    for (int i = i0 + lane; i < i1; i += 32)
      if (uint32_t(ids[i]) >= uint32_t(E)) p.slot[i] = -1;
  }
  if (mine == 0) return;
  int first = 0;  // pairs of this expert in the warps before, then in the places before
  for (int w = 0; w < warp; ++w) first += warp_count[w];
  for (int i = i0 + 4 * lane; i - 4 * lane < i1; i += 128) {
    const int4 d = load_ids(ids, i, i1, aligned);
    const int n = (d.x == e) + (d.y == e) + (d.z == e) + (d.w == e);
    if (!__any_sync(0xffffffffu, n)) continue;
    int scan = n;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, scan, x);
      if (lane >= x) scan += v;
    }
    int r = first + scan - n;
    if (d.x == e) p.slot[i] = base + moe_place(p, r++);
    if (d.y == e) p.slot[i + 1] = base + moe_place(p, r++);
    if (d.z == e) p.slot[i + 2] = base + moe_place(p, r++);
    if (d.w == e) p.slot[i + 3] = base + moe_place(p, r++);
    first += __shfl_sync(0xffffffffu, scan, 31);
  }
}

// y[t] = sum_j weights[t, j] * out[slot[t, j]] in fp32, rounded once.  Without
// slots, a pair's row is its own number (and counts if its id is an expert).
template <int DT>
__global__ void __launch_bounds__(256)
    moe_combine_kernel(const float* __restrict__ out, const int32_t* __restrict__ slot,
                       const int32_t* __restrict__ ids, int E, const float* __restrict__ weights,
                       int top_k, int64_t D, void* y) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t t = blockIdx.x;
  const int64_t d = (int64_t(blockIdx.y) * 256 + threadIdx.x) * 8;
  if (d >= D) return;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  constexpr int U = 4;  // rows in flight
  for (int j0 = 0; j0 < top_k; j0 += U) {
    int64_t r[U];
    float w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t p = t * top_k + j0 + u;
      r[u] = -1;
      if (j0 + u < top_k) {
        r[u] = slot != nullptr ? slot[p] : uint32_t(ids[p]) < uint32_t(E) ? p : -1;
        w[u] = weights[p];
      }
    }
    Raw8<LUTQ_FP32> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r[u] >= 0) raw[u] = load_raw8<LUTQ_FP32>(out, r[u] * D + d);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r[u] < 0) continue;
      float v[8];
      widen8<LUTQ_FP32>(raw[u], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += w[u] * v[i];
    }
  }
  store8<DT>(y, t * D + d, s);
}

// ------------------------------------------------------------------ host side

cudaError_t launch_mx_quantize(const void* x, int dtype, int64_t batch, int64_t items,
                               int64_t rows, int64_t K, int fmt, const int32_t* from,
                               const int32_t* to, int copies, void* packed, int32_t* dev_status,
                               int num_sms, cudaStream_t stream);

// Rows of all experts at most.  Tiles of 128: every pair, and each expert in
// use padded to 128.  Narrower tiles have room for T pairs or more, so the
// tiles that are not their expert's last are at most top_k.  (Both bounds for
// any T: the space for a batch also holds a smaller one.)
static int64_t moe_rows(int64_t T, int top_k, int E) {
  const int64_t pairs = T * top_k, used = std::min<int64_t>(E, pairs);
  return 128 * std::max(mx_ceil(pairs + 127 * used, 128), used + top_k);
}

struct MoeSpace {
  int64_t counts, bases, slot, xq, h, hq, out, bytes;
};
static MoeSpace moe_space(int64_t T, int top_k, int E, int64_t D, int64_t F, int fmt) {
  const int64_t cap = moe_rows(T, top_k, E);
  MoeSpace s;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += mx_ceil(bytes, 256) * 256;
    return here;
  };
  s.counts = take(4 * int64_t(E));
  s.bases = take(4 * int64_t(E));
  s.slot = take(4 * T * top_k);
  s.xq = take(mx_bytes(cap, D, fmt));
  s.h = take(2 * cap * F);
  s.hq = take(mx_bytes(cap, F, fmt));
  s.out = take(4 * cap * D);
  s.bytes = at;
  return s;
}
int64_t moe_workspace_bytes(int64_t T, int top_k, int E, int64_t D, int64_t F, int fmt) {
  return moe_space(T, top_k, E, D, F, fmt).bytes;
}

cudaError_t launch_mx_experts(const void* x, int dtype, int64_t T, const int32_t* ids,
                              const float* weights, int top_k, int E, const void* gate,
                              const void* up, const void* down, int fmt, int64_t D, int64_t F,
                              void* y, void* workspace, int32_t* dev_status, int num_sms,
                              cudaStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const MoeSpace s = moe_space(T, top_k, E, D, F, fmt);
  auto ints = [&](int64_t off) { return reinterpret_cast<int32_t*>(ws + off); };
  const int64_t cap = moe_rows(T, top_k, E);
  const int pairs = int(T * top_k);
  // pairs of a tile: an expert has T top_k / E on average, and no more than T
  // unless a token names it more than once (block pairs: whole runs of rows)
  const bool wide = mx_ceil(pairs, E) > kWidePairs && T > 32;
  const int nt = wide ? 128 : mx_tile_tokens(T);
  int nt_log2 = 4;
  while (1 << nt_log2 < nt) ++nt_log2;
  const MoePlan p = {ints(s.counts), ints(s.bases), ints(s.slot), nt_log2};
  // The pairs' rows stay in fp32 until they are summed.  (Rounded to bf16 they
  // would be half the bytes, and the sum off by up to 2^-8 of each of them.)
  auto combine = [&](const int32_t* slot) {
    const unsigned threads = unsigned(std::min<int64_t>(256, mx_ceil(D / 8, 32) * 32));
    auto go = [&](auto kernel) {
      return launch_pdl(kernel, dim3(unsigned(T), unsigned(mx_ceil(D, 2048))), dim3(threads), 0,
                        stream, reinterpret_cast<const float*>(ws + s.out), slot, ids, E, weights,
                        top_k, D, y);
    };
    if (dtype == LUTQ_BF16) return go(moe_combine_kernel<LUTQ_BF16>);
    if (dtype == LUTQ_FP16) return go(moe_combine_kernel<LUTQ_FP16>);
    return go(moe_combine_kernel<LUTQ_FP32>);
  };
  const int64_t small = fmt == LUTQ_MXFP4 ? kSmallPairsMx : kSmallPairsNv;
  if (mx_small_fits(pairs, E) && pairs <= small * std::min(E, pairs)) {
    // a handful of pairs an expert: quantized inside the products, three launches
    MxGemmArgs a = {};
    a.dev_status = dev_status;
    a.experts = E;
    a.x = x;
    a.x_dtype = dtype;
    a.y = ws + s.h;
    a.N = F;
    a.K = D;
    cudaError_t err = launch_mx_small(a, gate, up, fmt, kMxGateUp, ids, pairs, top_k, num_sms,
                                      stream);
    if (err != cudaSuccess) return err;
    // (nothing may come in between: this one reads ids and weights before it
    // waits for the launch before it, see launch_pdl)
    a.x = ws + s.h;
    a.x_dtype = LUTQ_BF16;
    a.y = ws + s.out;
    a.N = D;
    a.K = F;
    err = launch_mx_small(a, down, nullptr, fmt, kMxDown, ids, pairs, top_k, num_sms, stream);
    return err != cudaSuccess ? err : combine(nullptr);
  }
  const int64_t w1 = mx_bytes(F, D, fmt), w2 = mx_bytes(D, F, fmt);
  const int64_t used = std::min<int64_t>(E, pairs);  // experts in use at most
  CUtensorMap maps[4];
  std::memset(maps, 0, sizeof(maps));
  cudaError_t err;
  auto token_maps = [&](const void* rows, int64_t width) {
    const cudaError_t e = make_mx_map(&maps[2], rows, cap, width, 1, mx_bytes(cap, width, fmt), nt);
    return e != cudaSuccess
               ? e
               : make_mx_map(&maps[3], rows, cap, width, 1, mx_bytes(cap, width, fmt), 16);
  };

  auto plan = [&](auto kernel) {
    return launch_pdl(kernel, dim3(unsigned(E)), dim3(kPlanThreads), 0, stream, ids, pairs, E, p);
  };
  if (pairs <= kPlanAll) {
    err = plan(moe_plan_kernel<PLAN_ALL>);
  } else if ((err = plan(moe_plan_kernel<PLAN_COUNT>)) == cudaSuccess) {
    err = plan(moe_plan_kernel<PLAN_PLACE>);
  }
  if (err != cudaSuccess) return err;
  if ((err = launch_mx_quantize(x, dtype, 1, T, cap, D, fmt, nullptr, p.slot, top_k, ws + s.xq,
                                dev_status, num_sms, stream)) != cudaSuccess)
    return err;

  MxGemmArgs a = {};
  a.dev_status = dev_status;
  a.counts = p.counts;
  a.bases = p.bases;
  a.experts = E;
  a.M = cap;
  auto bytes = [](const void* q, int64_t off) { return static_cast<const uint8_t*>(q) + off; };
  a.a_scales[0] = bytes(gate, mx_scale_off(F, D));
  a.a_scales[1] = bytes(up, mx_scale_off(F, D));
  a.a_rows[0] = reinterpret_cast<const float*>(bytes(gate, mx_row_off(F, D, fmt)));
  a.a_rows[1] = reinterpret_cast<const float*>(bytes(up, mx_row_off(F, D, fmt)));
  a.a_stride = w1;
  a.b_scales = ws + s.xq + mx_scale_off(cap, D);
  a.b_rows = reinterpret_cast<const float*>(ws + s.xq + mx_row_off(cap, D, fmt));
  a.y = ws + s.h;
  a.N = F;
  a.K = D;
  a.chunks = int(mx_ceil(D, kMxChunk));
  a.mtiles = int(mx_ceil(F, 128));
  const bool packed_h = wide && fmt == LUTQ_MXFP4;
  if (wide) {
    if (packed_h) a.y = ws + s.hq;  // quantized by the product
    err = launch_mx_pair(a, gate, up, w1, ws + s.xq, cap, fmt, kMxGateUp,
                         (used + pairs / 128) * mx_ceil(F, 256), num_sms, stream);
  } else {
    if ((err = make_mx_map(&maps[0], gate, F, D, E, w1, 128)) != cudaSuccess) return err;
    if ((err = make_mx_map(&maps[1], up, F, D, E, w1, 128)) != cudaSuccess) return err;
    if ((err = token_maps(ws + s.xq, D)) != cudaSuccess) return err;
    err = launch_mx_gemm(maps, a, fmt, kMxGateUp, nt, (used + pairs / nt) * a.mtiles, num_sms,
                         stream);
  }
  if (err != cudaSuccess) return err;
  if (!packed_h &&
      (err = launch_mx_quantize(ws + s.h, LUTQ_BF16, 1, pairs, cap, F, fmt, p.slot, p.slot, 1,
                                ws + s.hq, dev_status, num_sms, stream)) != cudaSuccess)
    return err;

  a.a_scales[0] = a.a_scales[1] = bytes(down, mx_scale_off(D, F));
  a.a_rows[0] = a.a_rows[1] = reinterpret_cast<const float*>(bytes(down, mx_row_off(D, F, fmt)));
  a.a_stride = w2;
  a.b_scales = ws + s.hq + mx_scale_off(cap, F);
  a.b_rows = reinterpret_cast<const float*>(ws + s.hq + mx_row_off(cap, F, fmt));
  a.y = ws + s.out;
  a.y_dtype = LUTQ_FP32;
  a.N = D;
  a.K = F;
  a.chunks = int(mx_ceil(F, kMxChunk));
  a.mtiles = int(mx_ceil(D, 128));
  if (wide) {
    err = launch_mx_pair(a, down, nullptr, w2, ws + s.hq, cap, fmt, kMxDown,
                         (used + pairs / 256) * mx_ceil(D, 256), num_sms, stream);
  } else {
    if ((err = make_mx_map(&maps[0], down, D, F, E, w2, 128)) != cudaSuccess) return err;
    maps[1] = maps[0];
    if ((err = token_maps(ws + s.hq, F)) != cudaSuccess) return err;
    err = launch_mx_gemm(maps, a, fmt, kMxDown, nt, (used + pairs / nt) * a.mtiles, num_sms,
                         stream);
  }
  if (err != cudaSuccess) return err;
  return combine(p.slot);
}

}  // namespace lutq
