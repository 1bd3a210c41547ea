// Routing to experts: scores, selection and weights, one warp per token.
//
// The scores and every comparison are in 64 bits: which of two nearly equal
// experts wins is a discrete outcome, and 32-bit scores would decide it by the
// rounding of exp.  The arithmetic is small (E exponentials a token; a
// multiprocessor has half as many 64-bit as 32-bit lanes).  A lane keeps E / 32 scores as
// order-preserving 64-bit keys; the largest key of the warp takes three warp
// reductions (high word, low word, lowest expert), so ties go to the lowest
// expert whatever the order of arrival.
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
};

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
  double p[P];
  bool bad = false;
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = lane + 32 * i;
    float z = -INFINITY;
    if (e < E) {
      const int64_t at = t * E + e;
      if (a.dtype == LUTQ_FP32) z = static_cast<const float*>(a.logits)[at];
      else if (a.dtype == LUTQ_BF16) z = bf16_lo_to_f32(static_cast<const uint16_t*>(a.logits)[at]);
      else z = __half2float(static_cast<const __half*>(a.logits)[at]);
      bad |= isnan(z) || z == INFINITY;
      if (isnan(z)) z = -INFINITY;
    }
    p[i] = double(z);
    top = fmax(top, p[i]);
  }
  if (a.score == LUTQ_SCORE_SOFTMAX) {
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, x));
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
  const int per = E / a.groups;
  uint32_t kept = 0xffffffffu;
  if (a.groups > 1) {
    int pow2 = 2;
    while (pow2 < a.groups) pow2 *= 2;
    const int L = 32 / pow2, gr = lane / L;
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
      const bool in = p[i] >= 0.0 && (a.groups == 1 || ((kept >> (e / per)) & 1u));
      key[i] = in ? order_key(a.bias != nullptr ? p[i] + double(a.bias[e]) : p[i]) : kUnavailable;
    }
  }
  int mine = 0;          // lane j: the j-th choice
  double w = 0.0;
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
    if (lane == j) mine = won;
    const bool served = __any_sync(0xffffffffu, e == won && k > kUnavailable);
    if (lane == j) w = served ? ps[won] : 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (lane + 32 * i == won) key[i] = kTaken;
  }
  if (a.renormalize) {
    const double sum = warp_sum(lane < a.top_k ? w : 0.0);
    w = sum > 0.0 ? w / sum : 0.0;
  }
  if (lane < a.top_k) {
    a.ids[t * a.top_k + lane] = mine;
    a.weights[t * a.top_k + lane] = float(w * double(a.scale));
  }
  if (bad) report(a.dev_status, LUTQ_ERR_NONFINITE);
}

cudaError_t launch_route(const void* logits, int dtype, int64_t T, int E, const float* bias,
                         int score, int groups, int top_groups, int group_best, int top_k,
                         int renormalize, float scale, int32_t* ids, float* weights,
                         int32_t* dev_status, cudaStream_t stream) {
  RouteArgs a = {logits, bias,  ids,    weights,    dev_status, T,     dtype, E,
                 score,  groups, top_groups, group_best, top_k, renormalize, scale};
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
