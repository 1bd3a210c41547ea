// Microscaled 4-bit floating point: quantize, dequantize, pack (layout in
// lutq_mx.cuh).
//
// quantize is bound by memory: it reads 2 bytes a value (bf16) and writes
// 0.53 (mxfp4) or 0.56 (nvfp4).  A warp takes 256 values of one row at a time,
// 8 a lane, so that loads are 512 contiguous bytes, code stores 128 bytes, and
// a block's largest magnitude takes two (32 values) or one (16) shuffles.  A
// thread block takes rows p, p+1 and their partners 32, 64 and 96 below, whose
// scales are neighbours in the layout: its eight warps write whole 32-byte
// sectors of scales.  nvfp4 reads a row twice, first for the row's scale; the
// second read comes from L2 (8 rows a block, at most some tens of megabytes in
// flight).
#include <algorithm>

#include "lutq_mx.cuh"

namespace lutq {

constexpr int kMxWarps = 8;

// The row that warp w of block b of a row tile handles.
__device__ __forceinline__ int64_t mx_row_of(int b, int w) {
  return int64_t(b >> 4) * kMxRowTile + (b & 15) * 2 + (w & 1) + 32 * (w >> 1);
}
// Byte of row r's scales within a 512-byte block.
__device__ __forceinline__ int mx_scale_slot(int64_t r) {
  return int(r & 31) * 16 + int((r >> 5) & 3) * 4;
}

// Quantize one lane's 8 values; lanes 4i..4i+3 hold a block of 32 (mxfp4),
// 2i..2i+1 one of 16 (nvfp4).  Returns the codes; *scale the block's byte.
template <int FMT>
__device__ __forceinline__ uint32_t mx_quantize8(float (&v)[8], float g, float g_inv,
                                                 uint32_t* scale, bool* bad) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (FMT == LUTQ_MXFP4) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  if (m >= kInfBits) {  // a NaN or infinity: the block's scale is NaN
    *bad = true;
    *scale = FMT == LUTQ_MXFP4 ? 0xFFu : 0x7Fu;
    return 0u;
  }
  if constexpr (FMT == LUTQ_MXFP4) {
    *scale = e8m0_byte(m);
    const float inv = e8m0_inverse(*scale);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv;  // exact: a power of two
  } else {
    *scale = e4m3_byte(__uint_as_float(m) * g_inv / 6.0f);
    const float s = e4m3_value(*scale) * g;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = s > 0.f ? __fdiv_rn(v[j], s) : copysignf(0.f, v[j]);
  }
  return e2m1_x8(v);
}

// gather == nullptr: destination row r is source row r.  Otherwise row r is
// quantized from source row gather[r]; a negative entry leaves the row's
// bytes as they are (and `count`, if given, bounds the rows in use).
template <int FMT, int DT>
__global__ void __launch_bounds__(kMxWarps * 32)
    mx_quantize_kernel(const void* __restrict__ x, int64_t rows, int64_t K,
                       const int32_t* __restrict__ gather, const int32_t* __restrict__ count,
                       uint8_t* __restrict__ packed, int64_t x_stride, int64_t packed_stride,
                       int32_t* dev_status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = mx_row_of(blockIdx.x, warp);
  if (count != nullptr && int64_t(blockIdx.x >> 4) * kMxRowTile >= *count) return;
  const int64_t esize = DT == LUTQ_FP32 ? 4 : 2;
  const uint8_t* xm = static_cast<const uint8_t*>(x) + int64_t(blockIdx.z) * x_stride * esize;
  uint8_t* pm = packed + int64_t(blockIdx.z) * packed_stride;
  const int64_t chunks = mx_ceil(K, kMxChunk);
  // the zero padding below the last row of a tile is written too, except
  // among gathered rows, where nothing reads it
  int64_t src = r < rows ? r : -1;
  if (gather != nullptr) {
    src = r < rows ? gather[r] : -1;
    if (src < 0) return;
  }
  const uint8_t* xr = xm + src * K * esize;
  float g = 1.f, g_inv = 1.f;
  if (FMT == LUTQ_NVFP4 && src >= 0) {
    uint32_t m = 0;
    for (int64_t k = lane * 8; k < K; k += 256) {
      float v[8];
      load8<DT>(xr, k, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = abs_bits(v[j]);
        m = max(m, b < kInfBits ? b : 0u);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    g = nv_row_scale(m);
    g_inv = nv_row_scale_inverse(g);
    if (lane == 0 && blockIdx.y == 0)
      reinterpret_cast<float*>(pm + mx_row_off(rows, K, FMT))[r] = g;
  }
  bool bad = false;
  uint8_t* codes = pm + r * (K / 2);
  uint8_t* sc = pm + mx_scale_off(rows, K) +
                (r / kMxRowTile) * chunks * mx_chunk_bytes(FMT) + mx_scale_slot(r);
#pragma unroll 4
  for (int64_t c = blockIdx.y; c < chunks; c += gridDim.y) {
    const int64_t k = c * kMxChunk + lane * 8;
    uint32_t q = 0, s = 0;
    if (src >= 0) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (k < K) load8<DT>(xr, k, v);
      q = mx_quantize8<FMT>(v, g, g_inv, &s, &bad);
      if (k < K) *reinterpret_cast<uint32_t*>(codes + k / 2) = q;
      if (k >= K) s = 0;
    }
    // four scales of a block are one 32-bit word
    constexpr int L = FMT == LUTQ_MXFP4 ? 4 : 2;  // lanes per block
    uint32_t w = s << (8 * ((lane / L) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, L);
    w |= __shfl_xor_sync(0xffffffffu, w, 2 * L);
    if ((lane & (4 * L - 1)) == 0)
      *reinterpret_cast<uint32_t*>(sc + c * mx_chunk_bytes(FMT) + (lane / (4 * L)) * 512) = w;
  }
  if (bad) report(dev_status, LUTQ_ERR_NONFINITE);
}

// The values of 8 codes: (element * scale) * row scale, rounded once.
template <int FMT, int DT>
__global__ void __launch_bounds__(kMxWarps * 32)
    mx_dequantize_kernel(const uint8_t* __restrict__ packed, int64_t rows, int64_t K,
                         void* __restrict__ out, int64_t packed_stride) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = mx_row_of(blockIdx.x, warp);
  if (r >= rows) return;
  const uint8_t* pm = packed + int64_t(blockIdx.z) * packed_stride;
  const int64_t chunks = mx_ceil(K, kMxChunk);
  const uint8_t* codes = pm + r * (K / 2);
  const uint8_t* sc = pm + mx_scale_off(rows, K) +
                      (r / kMxRowTile) * chunks * mx_chunk_bytes(FMT) + mx_scale_slot(r);
  float g = 1.f;
  if (FMT == LUTQ_NVFP4) g = reinterpret_cast<const float*>(pm + mx_row_off(rows, K, FMT))[r];
  const int64_t base = (int64_t(blockIdx.z) * rows + r) * K;
  constexpr int L = FMT == LUTQ_MXFP4 ? 4 : 2;
#pragma unroll 4
  for (int64_t c = blockIdx.y; c < chunks; c += gridDim.y) {
    const int64_t k = c * kMxChunk + lane * 8;
    if (k >= K) continue;
    const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + k / 2);
    const uint32_t b = sc[c * mx_chunk_bytes(FMT) + (lane / (4 * L)) * 512 + ((lane / L) & 3)];
    const float s = FMT == LUTQ_MXFP4 ? e8m0_value(b) : e4m3_value(b);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e2m1_value((q >> (4 * j)) & 15u) * s * g;
    if constexpr (DT == LUTQ_FP32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + base + k);
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
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + base + k) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Codes (two a byte), row-major scale bytes and row scales into the layout.
template <int FMT>
__global__ void __launch_bounds__(kMxWarps * 32)
    mx_pack_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                   const float* __restrict__ row_scales, int64_t rows, int64_t K,
                   uint8_t* __restrict__ packed, int64_t packed_stride) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = mx_row_of(blockIdx.x, warp), z = blockIdx.z;
  uint8_t* pm = packed + z * packed_stride;
  const int64_t chunks = mx_ceil(K, kMxChunk), groups = K / mx_block(FMT);
  uint8_t* sc = pm + mx_scale_off(rows, K) +
                (r / kMxRowTile) * chunks * mx_chunk_bytes(FMT) + mx_scale_slot(r);
  if (FMT == LUTQ_NVFP4 && r < rows && lane == 0 && blockIdx.y == 0)
    reinterpret_cast<float*>(pm + mx_row_off(rows, K, FMT))[r] =
        row_scales == nullptr ? 1.f : row_scales[z * rows + r];
  constexpr int B = FMT == LUTQ_MXFP4 ? 2 : 4;  // 512-byte blocks per chunk
  for (int64_t c = blockIdx.y; c < chunks; c += gridDim.y) {
    const int64_t k = c * kMxChunk + lane * 8;
    if (r < rows && k < K)
      *reinterpret_cast<uint32_t*>(pm + r * (K / 2) + k / 2) =
          *reinterpret_cast<const uint32_t*>(codes + (z * rows + r) * (K / 2) + k / 2);
    if (lane < B) {
      uint32_t w = 0;
      for (int j = 0; j < 4; ++j) {
        const int64_t h = (c * B + lane) * 4 + j;
        if (r < rows && h < groups)
          w |= uint32_t(scales[(z * rows + r) * groups + h]) << (8 * j);
      }
      *reinterpret_cast<uint32_t*>(sc + c * mx_chunk_bytes(FMT) + lane * 512) = w;
    }
  }
}

// ------------------------------------------------------------------ host side

// Thread blocks along K: one row tile's blocks have 8 warps each, so a matrix
// of few rows is split along K until some hundreds of blocks run (nvfp4's row
// scale needs the whole row: no split).
static unsigned k_split(int64_t rows, int64_t K, int64_t batch, int num_sms) {
  const int64_t blocks = mx_ceil(rows, kMxRowTile) * 16 * batch;
  const int64_t want = mx_ceil(int64_t(num_sms) * 8, blocks);
  return unsigned(std::max<int64_t>(1, std::min<int64_t>(want, mx_ceil(K, kMxChunk))));
}

cudaError_t launch_mx_quantize(const void* x, int dtype, int64_t batch, int64_t rows, int64_t K,
                               int fmt, const int32_t* gather, const int32_t* count, void* packed,
                               int32_t* dev_status, int num_sms, cudaStream_t stream) {
  const dim3 grid(unsigned(mx_ceil(rows, kMxRowTile) * 16),
                  fmt == LUTQ_MXFP4 ? k_split(rows, K, batch, num_sms) : 1u, unsigned(batch));
  const int64_t xs = rows * K, ps = mx_bytes(rows, K, fmt);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kMxWarps * 32), 0, stream, x, rows, K, gather, count,
                      static_cast<uint8_t*>(packed), xs, ps, dev_status);
  };
  if (fmt == LUTQ_MXFP4) {
    if (dtype == LUTQ_BF16) return go(mx_quantize_kernel<LUTQ_MXFP4, LUTQ_BF16>);
    if (dtype == LUTQ_FP16) return go(mx_quantize_kernel<LUTQ_MXFP4, LUTQ_FP16>);
    return go(mx_quantize_kernel<LUTQ_MXFP4, LUTQ_FP32>);
  }
  if (dtype == LUTQ_BF16) return go(mx_quantize_kernel<LUTQ_NVFP4, LUTQ_BF16>);
  if (dtype == LUTQ_FP16) return go(mx_quantize_kernel<LUTQ_NVFP4, LUTQ_FP16>);
  return go(mx_quantize_kernel<LUTQ_NVFP4, LUTQ_FP32>);
}

cudaError_t launch_mx_dequantize(const void* packed, int64_t batch, int64_t rows, int64_t K,
                                 int fmt, void* out, int dtype, int num_sms,
                                 cudaStream_t stream) {
  const dim3 grid(unsigned(mx_ceil(rows, kMxRowTile) * 16), k_split(rows, K, batch, num_sms),
                  unsigned(batch));
  const int64_t ps = mx_bytes(rows, K, fmt);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kMxWarps * 32), 0, stream,
                      static_cast<const uint8_t*>(packed), rows, K, out, ps);
  };
  if (fmt == LUTQ_MXFP4) {
    if (dtype == LUTQ_BF16) return go(mx_dequantize_kernel<LUTQ_MXFP4, LUTQ_BF16>);
    if (dtype == LUTQ_FP16) return go(mx_dequantize_kernel<LUTQ_MXFP4, LUTQ_FP16>);
    return go(mx_dequantize_kernel<LUTQ_MXFP4, LUTQ_FP32>);
  }
  if (dtype == LUTQ_BF16) return go(mx_dequantize_kernel<LUTQ_NVFP4, LUTQ_BF16>);
  if (dtype == LUTQ_FP16) return go(mx_dequantize_kernel<LUTQ_NVFP4, LUTQ_FP16>);
  return go(mx_dequantize_kernel<LUTQ_NVFP4, LUTQ_FP32>);
}

cudaError_t launch_mx_pack(const uint8_t* codes, const uint8_t* scales, const float* row_scales,
                           int64_t batch, int64_t rows, int64_t K, int fmt, void* packed,
                           int num_sms, cudaStream_t stream) {
  const dim3 grid(unsigned(mx_ceil(rows, kMxRowTile) * 16), k_split(rows, K, batch, num_sms),
                  unsigned(batch));
  const int64_t ps = mx_bytes(rows, K, fmt);
  return launch_pdl(fmt == LUTQ_MXFP4 ? mx_pack_kernel<LUTQ_MXFP4> : mx_pack_kernel<LUTQ_NVFP4>,
                    grid, dim3(kMxWarps * 32), 0, stream, codes, scales, row_scales, rows, K,
                    static_cast<uint8_t*>(packed), ps);
}

}  // namespace lutq
