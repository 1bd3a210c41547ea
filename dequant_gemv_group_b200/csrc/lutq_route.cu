// Routing to experts: scores, selection and weights, one warp per token.
//
// The order of the scores is that of 64 bits: which of two nearly equal
// experts wins is a discrete outcome, and 32-bit scores alone would decide it
// by the rounding of exp.  64-bit exponentials of all scores are what this
// operator costs, so they are avoided where 32 bits suffice: the scores are
// selected in 32 bits first: the top_k, and those that are below by no more than
// both scores can be off.  Only these few get 64-bit scores, which give the
// weights, and the order where it is close.  Where 32 bits do not settle that
// much (a close call between groups, fewer experts available than asked for)
// the token is routed again with 64-bit scores.
//
// A lane holds every 32nd expert's score.  The largest score of the warp, and
// the lowest expert that has it, take two warp reductions of 32-bit keys
// (three for 64-bit ones), so ties go to the lowest expert.
#include <algorithm>
#include <cmath>

#include "lutq_mx.cuh"

namespace lutq {

constexpr int kRouteWarps = 4;

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int32_t* dev_status;
  int64_t T;
  int dtype, E, score, groups, top_groups, group_best, top_k, renormalize;
  float scale;
  int per;             // experts of a group
  uint32_t per_magic;  // ceil(2^20 / per): e / per = e * magic >> 20 for e < 1024, per <= 512
  int group_lanes;     // log2 of the lanes that share a group
};

__device__ __forceinline__ int group_of(const RouteArgs& a, int e) {
  return int(uint32_t(e) * a.per_magic >> 20);
}

// Doubles to unsigned keys in the same order, all above 1.
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t b = uint64_t(__double_as_longlong(v + 0.0));  // -0 becomes +0
  return (b >> 63) ? ~b : b | (uint64_t(1) << 63);
}
constexpr uint64_t kTaken = 0, kUnavailable = 1;

// The largest key of the warp and the lowest index among its holders.
__device__ __forceinline__ int warp_argmax(uint64_t key, int index) {
  const uint32_t hi = uint32_t(key >> 32), lo = uint32_t(key);
  const uint32_t mh = __reduce_max_sync(0xffffffffu, hi);
  const uint32_t ml = __reduce_max_sync(0xffffffffu, hi == mh ? lo : 0u);
  return int(__reduce_min_sync(0xffffffffu, hi == mh && lo == ml ? uint32_t(index) : 0xffffffffu));
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int x = 16; x; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
  return v;
}

// Floats to unsigned keys in the same order; 0 stands for "taken".  The lowest
// bits, log2 P of them, are given up for the number of the score in its lane.
__device__ __forceinline__ uint32_t order_key32(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value32(uint32_t k) {
  // (below the key of the lowest float: -infinity, whatever its low bits)
  return k < 0x00800000u ? -INFINITY : __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}
// Whether 32-bit scores tell the order of the exact ones.  `base` bounds the
// error of p: sigmoid, 1 / (1 + e) with e off by (2 + 1.2 |z|) ulp and a
// division by 2 ulp, in all below 4e-7; softmax, e off by 6 2^-24, a sum of P
// and 5 additions, a division and a product, below (P + 20) 2^-24.  `rel`
// times the score bounds that of the addition of the bias and of a key's lost
// bits.
struct Error32 {
  float base, rel;
};
__device__ __forceinline__ bool clearly_above(float a, float b, Error32 e) {
  if (b == -INFINITY) return a > -INFINITY;  // nothing available there
  return a - b > 2.f * e.base + e.rel * (fabsf(a) + fabsf(b));
}

// The selection in 32 bits.  Lane j < n receives the expert with the j-th
// largest 32-bit score (j alone where the order is clear); the top_k largest
// exact scores are certainly among these n.  Returns n, or 0 if 32 bits do not
// tell: which groups stay, fewer available than asked for, too many close.
template <int P>
__device__ __forceinline__ int route_select32(const RouteArgs& a, const float (&z)[P], float top,
                                               float* cs, int lane, int* mine,
                                              bool* ordered) {
  const int E = a.E;
  const float base = a.score == LUTQ_SCORE_SOFTMAX ? float(P + 20) * 0x1p-24f : 4e-7f;
  const Error32 score_error = {base, float(P + 1) * 0x1p-23f};
  float c[P], bias[P];
#pragma unroll
  for (int i = 0; i < P; ++i)
    bias[i] = a.bias != nullptr && lane + 32 * i < E ? a.bias[lane + 32 * i] : 0.f;
  if (a.score == LUTQ_SCORE_SOFTMAX) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      c[i] = z[i] > -INFINITY ? __expf(z[i] - top) : 0.f;
      sum += c[i];
    }
    if (a.bias != nullptr) {  // (without one the exponentials have the order)
#pragma unroll
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      sum = 1.f / sum;
#pragma unroll
      for (int i = 0; i < P; ++i) c[i] *= sum;
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] = __fdividef(1.f, 1.f + __expf(-z[i]));
  }
#pragma unroll
  for (int i = 0; i < P; ++i) c[i] = z[i] > -INFINITY ? c[i] + bias[i] : -INFINITY;
  if (a.groups > 1) {
    bool clear = true;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 32 * i < E) cs[lane + 32 * i] = c[i];
    __syncwarp();
    const int L = 1 << a.group_lanes, gr = lane >> a.group_lanes;
    float b0 = -INFINITY, b1 = -INFINITY;  // the two best
    if (gr < a.groups) {
      const float* cg = cs + gr * a.per;
      for (int j = lane & (L - 1); j < a.per; j += L) {
        const float v = cg[j];
        b1 = fmaxf(b1, fminf(b0, v));
        b0 = fmaxf(b0, v);
      }
    }
    for (int x = 1; x < L; x *= 2) {
      const float o0 = __shfl_xor_sync(0xffffffffu, b0, x);
      const float o1 = __shfl_xor_sync(0xffffffffu, b1, x);
      b1 = fmaxf(fmaxf(b1, o1), fminf(b0, o0));
      b0 = fmaxf(b0, o0);
    }
    const bool two = a.group_best == 2 && b1 > -INFINITY;
    const float best = two ? b0 + b1 : b0;
    // How far off: by both scores' p, and by the roundings of both biased scores
    // and of their sum, each below 2^-24 of itself.  The scores may cancel, so it
    // is their magnitudes that count.  (-infinity: exact)
    const float off =
        best > -INFINITY ? 2.f * base + 0x1p-22f * (fabsf(b0) + (two ? fabsf(b1) : 0.f)) : 0.f;
    uint32_t gk = gr < a.groups && (lane & (L - 1)) == 0 ? order_key32(best) : 0u;
    const bool scored = gk != 0u;
    uint32_t kept = 0;
    for (int i = 0; i < a.top_groups; ++i) {
      const uint32_t last = __reduce_max_sync(0xffffffffu, gk);
      // (equal ones leave together; then the order is not clear)
      const uint32_t who = __ballot_sync(0xffffffffu, gk == last);
      clear = clear && (who & (who - 1u)) == 0u;
      kept |= 1u << ((__ffs(who) - 1) >> a.group_lanes);
      if (gk == last) gk = 0u;
    }
    // the lowest that a kept group can be, the highest that another can be
    const uint32_t low = __reduce_min_sync(
        0xffffffffu, scored && gk == 0u ? order_key32(best - off) : 0xffffffffu);
    const uint32_t high = __reduce_max_sync(0xffffffffu, gk != 0u ? order_key32(best + off) : 0u);
    if (!clear || low <= high) return 0;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (!((kept >> group_of(a, lane + 32 * i)) & 1u)) c[i] = -INFINITY;
  }
  uint32_t key[P];
#pragma unroll
  for (int i = 0; i < P; ++i)
    key[i] = lane + 32 * i < E ? (order_key32(c[i]) & ~uint32_t(P - 1)) | uint32_t(i) : 0u;
  float mine_v = 0.f, kth = 0.f;  // lane j: the j-th score; the top_k-th
  int n = 0;
  for (;; ++n) {
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < P; ++i) m = max(m, key[i]);
    const uint32_t k = __reduce_max_sync(0xffffffffu, m);
    const float v = key_value32(k);
    if (n < a.top_k) {
      if (v == -INFINITY) return 0;
      kth = v;
    } else {
      if (clearly_above(kth, v, score_error)) break;
      if (n == 32) return 0;
    }
    const int w = __ffs(__ballot_sync(0xffffffffu, m == k)) - 1;
    if (lane == n) {
      mine_v = v;
      *mine = w + 32 * int(k & uint32_t(P - 1));
    }
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = key[i] == k && lane == w ? 0u : key[i];
  }
  const float before = __shfl_up_sync(0xffffffffu, mine_v, 1);
  *ordered = __all_sync(0xffffffffu, lane == 0 || lane >= n ||
                                         clearly_above(before, mine_v, score_error));
  return n;  // the same in all lanes
}

__device__ __forceinline__ float load_logit(const RouteArgs& a, int64_t at) {
  if (a.dtype == LUTQ_FP32) return static_cast<const float*>(a.logits)[at];
  if (a.dtype == LUTQ_BF16) return bf16_lo_to_f32(static_cast<const uint16_t*>(a.logits)[at]);
  return __half2float(static_cast<const __half*>(a.logits)[at]);
}

// The selection in 64 bits: lane j receives the j-th choice and its score.
struct Choice {
  double w;
  int mine;
};
template <int P>
__device__ __noinline__ Choice route_select64(const RouteArgs& a, int64_t t, float topf,
                                              double* ps, int lane) {
  const int E = a.E;
  Choice out = {0.0, 0};
  double p[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float z = -INFINITY;
    if (lane + 32 * i < E) z = load_logit(a, t * E + lane + 32 * i);
    p[i] = isnan(z) ? -INFINITY : double(z);
  }
  if (a.score == LUTQ_SCORE_SOFTMAX) {
    const double top = double(topf);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (p[i] == -INFINITY) {
        p[i] = -1.0;
      } else {
        p[i] = p[i] == top ? 1.0 : exp(p[i] - top);
        sum += p[i];
      }
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (p[i] >= 0.0) p[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = p[i] == -INFINITY ? -1.0 : 1.0 / (1.0 + exp(-p[i]));
  }
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (lane + 32 * i < E) ps[lane + 32 * i] = p[i];
  __syncwarp();

  // groups: the sum of a group's best scores; the best groups stay
  const int per = a.per;
  uint32_t kept = 0xffffffffu;
  if (a.groups > 1) {
    const int L = 1 << a.group_lanes, gr = lane >> a.group_lanes;
    double b0 = -INFINITY, b1 = -INFINITY;  // the two best
    if (gr < a.groups) {
      for (int j = lane % L; j < per; j += L) {
        const int e = gr * per + j;
        const double q = ps[e];
        if (q < 0.0) continue;
        const double c = a.bias != nullptr ? q + double(a.bias[e]) : q;
        b1 = fmax(b1, fmin(b0, c));
        b0 = fmax(b0, c);
      }
    }
    for (int x = 1; x < L; x *= 2) {
      const double o0 = __shfl_xor_sync(0xffffffffu, b0, x);
      const double o1 = __shfl_xor_sync(0xffffffffu, b1, x);
      b1 = fmax(fmax(b1, o1), fmin(b0, o0));
      b0 = fmax(b0, o0);
    }
    const double best = a.group_best == 2 && b1 > -INFINITY ? b0 + b1 : b0;
    uint64_t key = gr < a.groups && lane % L == 0 ? order_key(best) : kTaken;
    kept = 0;
    for (int i = 0; i < a.top_groups; ++i) {
      const int g = warp_argmax(key, gr);
      kept |= 1u << g;
      if (g == gr) key = kTaken;
    }
  }

  uint64_t key[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 32 * i;
    key[i] = kTaken;
    if (e < E) {
      const bool in = p[i] >= 0.0 && (a.groups == 1 || ((kept >> group_of(a, e)) & 1u));
      key[i] = in ? order_key(a.bias != nullptr ? p[i] + double(a.bias[e]) : p[i]) : kUnavailable;
    }
  }
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t k = kTaken;
    int e = E;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (key[i] > k) {
        k = key[i];
        e = lane + 32 * i;
      }
    const int won = warp_argmax(k, e);
    if (lane == j) out.mine = won;
    const bool served = __any_sync(0xffffffffu, e == won && k > kUnavailable);
    if (lane == j) out.w = served ? ps[won] : 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 32 * i == won) key[i] = kTaken;
  }
  return out;
}

// P: scores a lane holds (E <= 32 P)
template <int P>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ double route_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = int64_t(blockIdx.x) * kRouteWarps + warp;
  if (t >= a.T) return;
  double* ps = route_smem + warp * a.E;  // the token's scores; -1: not available
  const int E = a.E;
  float z[P];
  bool bad = false;
  float topf = -INFINITY;
  const int64_t first = t * E + lane;
#pragma unroll
  for (int i = 0; i < P; ++i) z[i] = -INFINITY;
  if (a.dtype == LUTQ_FP32) {
    const float* p = static_cast<const float*>(a.logits) + first;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 32 * i < E) z[i] = p[32 * i];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.logits) + first;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 32 * i < E)
        z[i] = a.dtype == LUTQ_BF16 ? bf16_lo_to_f32(p[32 * i])
                                    : __half2float(__ushort_as_half(p[32 * i]));
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    bad |= !(z[i] < INFINITY);  // NaN, too
    if (isnan(z[i])) z[i] = -INFINITY;
    topf = fmaxf(topf, z[i]);
  }
  if (a.score == LUTQ_SCORE_SOFTMAX) {
#pragma unroll
    for (int x = 16; x; x >>= 1) topf = fmaxf(topf, __shfl_xor_sync(0xffffffffu, topf, x));
  }
  if (bad) report(a.dev_status, LUTQ_ERR_NONFINITE);
  int mine = 0, rank = lane;  // an expert, its place among the chosen, its score
  double w = 0.0;
  int n = 0;
  if (!__any_sync(0xffffffffu, bad)) {
    bool ordered = true;
    n = route_select32<P>(a, z, topf, reinterpret_cast<float*>(ps), lane, &mine, &ordered);
    if (lane < n) {
      const double v = double(load_logit(a, t * E + mine));
      w = a.score == LUTQ_SCORE_SOFTMAX ? exp(v - double(topf)) : 1.0 / (1.0 + exp(-v));
    }
    // a softmax's sum, unless it cancels (renormalised, and no bias to add to p)
    if (n > 0 && a.score == LUTQ_SCORE_SOFTMAX &&
        (!a.renormalize || (!ordered && a.bias != nullptr))) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (z[i] > -INFINITY) sum += exp(double(z[i]) - double(topf));
      w /= warp_sum(sum);
    }
    if (n > 0 && !ordered) {
      // the exact order of the few: how many come before this one
      const double c = w + (a.bias != nullptr && lane < n ? double(a.bias[mine]) : 0.0);
      rank = 0;
      for (int j = 0; j < n; ++j) {
        const double cj = __shfl_sync(0xffffffffu, c, j);
        const int ej = __shfl_sync(0xffffffffu, mine, j);
        rank += cj > c || (cj == c && ej < mine);
      }
      if (lane >= n) rank = 32;
    }
    __syncwarp();
  }
  if (n == 0) {
    const Choice c = route_select64<P>(a, t, topf, ps, lane);
    mine = c.mine;
    w = c.w;
  }
  const bool in = rank < a.top_k;
  if (a.renormalize) {
    const double sum = warp_sum(in ? w : 0.0);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (in) {
    a.ids[t * a.top_k + rank] = mine;
    a.weights[t * a.top_k + rank] = float(w * double(a.scale));
  }
}

cudaError_t launch_route(const void* logits, int dtype, int64_t T, int E, const float* bias,
                         int score, int groups, int top_groups, int group_best, int top_k,
                         int renormalize, float scale, int32_t* ids, float* weights,
                         int32_t* dev_status, cudaStream_t stream) {
  RouteArgs a = {logits, bias,       ids,        weights, dev_status,  T,
                 dtype,  E,          score,      groups,  top_groups,  group_best,
                 top_k,  renormalize, scale,     E / groups, 0,        5};
  a.per_magic = uint32_t(mx_ceil(int64_t(1) << 20, a.per));
  while ((32 >> a.group_lanes) < groups) --a.group_lanes;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(mx_ceil(T, kRouteWarps)));
  cfg.blockDim = dim3(kRouteWarps * 32);
  cfg.dynamicSmemBytes = size_t(kRouteWarps) * size_t(E) * sizeof(double);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (E <= 32) return cudaLaunchKernelEx(&cfg, route_kernel<1>, a);
  if (E <= 64) return cudaLaunchKernelEx(&cfg, route_kernel<2>, a);
  if (E <= 128) return cudaLaunchKernelEx(&cfg, route_kernel<4>, a);
  if (E <= 256) return cudaLaunchKernelEx(&cfg, route_kernel<8>, a);
  if (E <= 512) return cudaLaunchKernelEx(&cfg, route_kernel<16>, a);
  return cudaLaunchKernelEx(&cfg, route_kernel<32>, a);
}

}  // namespace lutq
