// Microscaled 4-bit floating point: the packed layout and the conversions
// shared by the quantizer, the products and the experts' layer.
//
// An element is E2M1 (sign, levels 0 .5 1 1.5 2 3 4 6); a block of consecutive
// elements along K shares a scale byte: mxfp4 has blocks of 32 and E8M0 scales
// (2^(byte - 127), 0xFF = NaN), nvfp4 blocks of 16, E4M3 scales and one fp32
// scale per row.
//
// Packed layout of a matrix of `rows` x K (K % 32 == 0):
//   codes   rows * K / 2 bytes, row-major, element 2i in the low nibble;
//           padded to 128 bytes;
//   scales  [ceil(rows/128)][ceil(K/256)] chunks, each of 2 (mxfp4) or 4
//           (nvfp4) blocks of 512 bytes; a block holds four scales along K of
//           each of 128 rows: row r, scale j at byte 16 (r % 32) + 4 (r / 32)
//           + j.  Tensor memory takes such a block in one copy (32 lanes of
//           four 32-bit columns).  Bytes of rows and columns beyond the
//           matrix are zero, so that a padded product adds 0 * 0;
//   rows    nvfp4: fp32 [rows], padded to 128 bytes.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_fp16.h>

#include "lutq_common.cuh"

namespace lutq {

constexpr int kMxChunk = 256;     // elements of K per scale chunk (128 bytes of codes)
constexpr int kMxRowTile = 128;   // rows per scale block

__host__ __device__ constexpr int mx_block(int fmt) { return fmt == LUTQ_MXFP4 ? 32 : 16; }
__host__ __device__ constexpr int mx_chunk_bytes(int fmt) {
  return fmt == LUTQ_MXFP4 ? 1024 : 2048;
}
__host__ __device__ constexpr int64_t mx_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ constexpr int64_t mx_scale_off(int64_t rows, int64_t K) {
  return mx_ceil(rows * (K / 2), 128) * 128;
}
__host__ __device__ constexpr int64_t mx_row_off(int64_t rows, int64_t K, int fmt) {
  return mx_scale_off(rows, K) +
         mx_ceil(rows, kMxRowTile) * mx_ceil(K, kMxChunk) * mx_chunk_bytes(fmt);
}
__host__ __device__ constexpr int64_t mx_bytes(int64_t rows, int64_t K, int fmt) {
  return mx_row_off(rows, K, fmt) + (fmt == LUTQ_NVFP4 ? mx_ceil(rows, 32) * 128 : 0);
}

// Eight floats to eight E2M1 codes (round to nearest, ties to the even code,
// saturating at 6), element 0 in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1_x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The values of eight codes, element 0 in the lowest nibble.
__device__ __forceinline__ void e2m1_values8(uint32_t q, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

// One float >= 0 to E4M3 (round to nearest even, saturating at 448).
__device__ __forceinline__ uint32_t e4m3_byte(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return r & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(uint16_t(b)));
  return __half2float(__ushort_as_half(uint16_t(h2)));
}

// E8M0: the scale's exponent byte from the block's largest magnitude (as fp32
// bits): floor(log2 amax) - 2 + 127, at least 0 (a subnormal amax is far below
// 2^-125).
__device__ __forceinline__ uint32_t e8m0_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e > 2u ? e - 2u : 0u;
}
// 2^(127 - byte) for byte <= 252: the exact reciprocal of the scale.
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  // 2^-127 is subnormal; 0xFF stands for NaN
  return byte == 0u ? __uint_as_float(0x00400000u)
                    : (byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(byte << 23));
}

// nvfp4's row scale: 2^(floor(log2 m) - 10) of the row's largest finite
// magnitude m (1 for a row of zeros), at least 2^-126.  Then m / 6 / g lies in
// [170, 342), inside E4M3's range.  A power of two keeps s * g, m / g and so
// every rounding decision on 16-bit inputs exact in fp32.
__device__ __forceinline__ float nv_row_scale(uint32_t max_bits) {
  if (max_bits == 0u) return 1.f;
  const uint32_t e = max_bits >> 23;
  return __uint_as_float((e > 11u ? e - 10u : 1u) << 23);
}
__device__ __forceinline__ float nv_row_scale_inverse(float g) {
  return __uint_as_float((254u - (__float_as_uint(g) >> 23)) << 23);
}

constexpr uint32_t kInfBits = 0x7f800000u;

// The same eight values as loaded: 16-bit pairs in four words, or fp32 in eight.
template <int DT>
struct Raw8 {
  uint32_t w[DT == LUTQ_FP32 ? 8 : 4];
};
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const void* base, int64_t i) {
  Raw8<DT> r;
  if constexpr (DT == LUTQ_FP32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
    const uint4 a = p[0], b = p[1];
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
  }
  return r;
}
template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < (DT == LUTQ_FP32 ? 8 : 4); ++j) {
    if constexpr (DT == LUTQ_FP32) {
      v[j] = __uint_as_float(r.w[j]);
    } else if constexpr (DT == LUTQ_BF16) {
      v[2 * j] = bf16_lo_to_f32(r.w[j]);
      v[2 * j + 1] = bf16_hi_to_f32(r.w[j]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[j]));
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
}
// The largest magnitude as the type's own bits (16-bit types: two at a time, by
// maxima that keep a NaN; its bits, like an infinity's, are the largest).
template <int DT>
__device__ __forceinline__ uint32_t max_raw8(const Raw8<DT>& r) {
  if constexpr (DT == LUTQ_FP32) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, r.w[j] & 0x7fffffffu);
    return m;
  } else {
    using T2 = std::conditional_t<DT == LUTQ_BF16, __nv_bfloat162, __half2>;
    T2 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __habs2(*reinterpret_cast<const T2*>(&r.w[j]));
    const T2 x = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    const uint32_t m = *reinterpret_cast<const uint32_t*>(&x) & 0x7fff7fffu;
    return max(m & 0xffffu, m >> 16);
  }
}
// Those bits as fp32 bits (an infinity or NaN stays one), and their limit.
template <int DT>
__device__ __forceinline__ uint32_t max_bits_f32(uint32_t m) {
  if constexpr (DT == LUTQ_FP32) return m;
  if constexpr (DT == LUTQ_BF16) return m << 16;
  return __float_as_uint(__half2float(__ushort_as_half(uint16_t(m))));
}
template <int DT>
__host__ __device__ constexpr uint32_t raw_inf() {
  return DT == LUTQ_FP32 ? 0x7f800000u : DT == LUTQ_BF16 ? 0x7f80u : 0x7c00u;
}

// Quotients for a rounding decision, without a division.  Where x and s have
// few bits, x / s is either exactly halfway between two neighbouring results
// or at least 2^-15 (relative) away from that: fp16 x (11 bits), s of 4 bits,
// halfway points of 3 for the levels; x / 6 and halfway points of 5 bits for
// E4M3.  A product with the approximate reciprocal is off by less than 2^-22;
// rounded to 17 bits it is halfway exactly when the quotient is, and otherwise
// on the same side.  (A division costs five times as much.  fp32 inputs have
// no such gap and are divided.)
__device__ __forceinline__ float snap17(float v) {
  return __uint_as_float((__float_as_uint(v) + 0x40u) & 0xffffff80u);
}
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// nvfp4: the scale byte of a block with largest magnitude m (fp32 bits).
template <int DT>
__device__ __forceinline__ uint32_t nv_scale_byte(uint32_t m, float g_inv) {
  const float t = __uint_as_float(m) * g_inv;
  return e4m3_byte(DT == LUTQ_FP32 ? t / 6.0f : snap17(t * (1.0f / 6.0f)));
}
// Eight values to their codes, s the block's scale (nvfp4) or unused.
template <int FMT, int DT>
__device__ __forceinline__ uint32_t mx_codes8(float (&v)[8], uint32_t scale, float g,
                                              float g_inv) {
  if constexpr (FMT == LUTQ_MXFP4) {
    const float inv = e8m0_inverse(scale);
    const uint64_t inv2 = pack2(inv, inv);
#pragma unroll
    for (int j = 0; j < 8; j += 2)  // exact: a power of two
      unpack2(mul2(pack2(v[j], v[j + 1]), inv2), v[j], v[j + 1]);
  } else {
    const float s = e4m3_value(scale);
    if constexpr (DT == LUTQ_FP32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = s > 0.f ? __fdiv_rn(v[j], s * g) : copysignf(0.f, v[j]);
    } else {
      // rows below 2^-100: 1 / (s g) may pass fp32's range; both sides times 2^64
      if (g_inv >= 0x1p110f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= 0x1p64f;
        g *= 0x1p64f;
        g_inv *= 0x1p-64f;
      }
      // a quotient r and one correction by its remainder x - r (s g): exact
      // where the quotient has few bits, as at a halfway point (the packed
      // multiply-adds are cheaper than two integer operations of snap17).
      // Computed as -(x / (s g)), so that a zero keeps its sign: the codes'
      // signs are turned back together.  (s = 0: every quotient is a zero.)
      const float m = s > 0.f ? rcp_approx(s) * -g_inv : -0.f, d = s * g;
      const uint64_t m2 = pack2(m, m), d2 = pack2(d, d);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint64_t x2 = pack2(v[j], v[j + 1]), r2 = mul2(x2, m2);
        unpack2(fma2(fma2(r2, d2, x2), m2, r2), v[j], v[j + 1]);
      }
      return e2m1_x8(v) ^ 0x88888888u;
    }
  }
  return e2m1_x8(v);
}

// silu(g) * u of a hidden value, the same for every batch size: with t =
// exp(-|g|), g / (1 + t) or g t / (1 + t), whose divisor lies in [1, 2], so that
// the quotient needs no special cases: a product with the approximate
// reciprocal and one correction by its remainder.  exp is off by at most 2 units
// of 2^-23 (in t and 1 + t together less than that), the four roundings by 2^-24
// each: less than 2^-21 in all, before the rounding to bf16.  (The fast
// exponential's error grows with |g|, to 2^-18 at -88, and the fast division
// gives 0 for a divisor above 2^126: hidden values moved by a bf16 step, or
// became 0.)
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float t = expf(-fabsf(g)), d = 1.f + t, r = rcp_approx(d);
  const float n = g < 0.f ? g * t : g, q = n * r;
  return fmaf(fmaf(-q, d, n), r, q) * u;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Value v rounded once to the output type, at element i of y.
template <int DT>
__device__ __forceinline__ void store1(void* y, int64_t i, float v) {
  if constexpr (DT == LUTQ_FP32) {
    static_cast<float*>(y)[i] = v;
  } else if constexpr (DT == LUTQ_BF16) {
    static_cast<uint16_t*>(y)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  } else {
    static_cast<uint16_t*>(y)[i] = __half_as_ushort(__float2half_rn(v));
  }
}

// The largest finite magnitude of eight values, as fp32 bits.
template <int DT>
__device__ __noinline__ uint32_t finite_max8(const Raw8<DT> raw) {
  float v[8];
  widen8<DT>(raw, v);
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]) < kInfBits ? abs_bits(v[j]) : 0u);
  return m;
}

// Quantize a lane's 8 of a warp's 256 values: lanes 4i..4i+3 hold a block of 32
// (mxfp4), 2i..2i+1 one of 16 (nvfp4).  Returns the lane's codes; *word: the
// scale bytes of the four neighbouring blocks that a word of the layout holds.
template <int FMT, int DT>
__device__ __forceinline__ uint32_t mx_quantize_lane(const Raw8<DT>& raw, float g, float g_inv,
                                                     int lane, uint32_t* word, bool* bad) {
  constexpr int L = FMT == LUTQ_MXFP4 ? 4 : 2;  // lanes per block
  uint32_t m = max_raw8<DT>(raw);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (FMT == LUTQ_MXFP4) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  uint32_t scale, codes = 0u;
  if (m >= raw_inf<DT>()) {  // a NaN or infinity: the block's scale is NaN
    *bad = true;
    scale = FMT == LUTQ_MXFP4 ? 0xFFu : 0x7Fu;
  } else {
    m = max_bits_f32<DT>(m);
    scale = FMT == LUTQ_MXFP4 ? e8m0_byte(m) : nv_scale_byte<DT>(m, g_inv);
    float v[8];
    widen8<DT>(raw, v);
    codes = mx_codes8<FMT, DT>(v, scale, g, g_inv);
  }
  uint32_t w = scale << (8 * ((lane / L) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, L);
  w |= __shfl_xor_sync(0xffffffffu, w, 2 * L);
  *word = w;
  return codes;
}

// Eight values rounded once to the output type, from element i (a multiple of
// 8, in a 16-byte aligned y).
template <int DT>
__device__ __forceinline__ void store8(void* y, int64_t i, const float (&v)[8]) {
  if constexpr (DT == LUTQ_FP32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(y) + i);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == LUTQ_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Launch with the next kernel of the stream allowed to start early: every
// kernel of this family waits for the one before it (griddepcontrol.wait)
// before it reads or writes anything.  One exception: the down product of few
// tokens reads ids, weights and their scales before its wait.  It may only be
// launched straight after the gate and up product of the same call, which lets
// it start (launch_dependents) after its own wait for all that came before.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

}  // namespace lutq
