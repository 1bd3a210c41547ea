// Microscaled 4-bit floating point: quantize, dequantize, pack (layout in
// lutq_mx.cuh).
//
// Both directions are bound by memory: quantize reads 2 bytes a value (bf16)
// and writes 0.53 (mxfp4) or 0.56 (nvfp4), dequantize the reverse.  A warp
// takes 256 values of a row at a time, 8 a lane, so that value accesses are
// 512 contiguous bytes, code accesses 128, and a block's largest magnitude
// takes two (32 values) or one (16) shuffles; several such loads are issued
// before the first is used.  Many rows: a warp takes a row; the eight warps of
// a block take rows p, p+1 and their partners 32, 64 and 96 below, whose
// scales are neighbours in the layout, and so write whole 32-byte sectors of
// scales.  Few rows: the block's warps share a row.  nvfp4 reads a row twice,
// first for the row's scale; the second read comes from L2.
#include <algorithm>

#include "lutq_mx.cuh"

namespace lutq {

constexpr int kMxWarps = 8;
constexpr int kMxBatch = 4;  // loads of a lane in flight

// The row that warp w of block b of a row tile handles.
__device__ __forceinline__ int64_t mx_row_of(int b, int w) {
  return int64_t(b >> 4) * kMxRowTile + (b & 15) * 2 + (w & 1) + 32 * (w >> 1);
}
// Byte of row r's scales within a 512-byte block.
__device__ __forceinline__ int mx_scale_slot(int64_t r) {
  return int(r & 31) * 16 + int((r >> 5) & 3) * 4;
}

// WPR warps share a row.  Not LISTED: row r is source and destination row r,
// and the zero padding below the last row of a tile is written too.  LISTED:
// item r reads source row from[r] (or r, if from is null) and goes to the
// `copies` rows to[copies * r ...]; a negative entry is skipped, and nothing
// else is written.
template <int FMT, int DT, int WPR, bool LISTED>
__global__ void __launch_bounds__(kMxWarps * 32, WPR == 1 && DT != LUTQ_FP32 ? 4 : 1)
    mx_quantize_kernel(const void* __restrict__ x, int64_t items, int64_t rows, int64_t K,
                       const int32_t* __restrict__ from, const int32_t* __restrict__ to,
                       int copies, uint8_t* __restrict__ packed, int64_t x_stride,
                       int64_t packed_stride, int32_t* dev_status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t row_max[kMxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = WPR == kMxWarps ? blockIdx.x
                       : LISTED        ? int64_t(blockIdx.x) * kMxWarps + warp
                                       : mx_row_of(blockIdx.x, warp);
  constexpr int64_t esize = DT == LUTQ_FP32 ? 4 : 2;
  int64_t src = item < items ? item : -1;
  if (LISTED) {
    if (item >= items) return;
    if (from != nullptr) src = from[item];
    if (src < 0) return;  // (the whole block, where its warps share the row)
  }
  const int to_lane = LISTED && lane < copies ? to[item * copies + lane] : -1;
  const uint8_t* xr = static_cast<const uint8_t*>(x) +
                      (int64_t(blockIdx.z) * x_stride + src * K + lane * 8) * esize;
  uint8_t* pm = packed + int64_t(blockIdx.z) * packed_stride;
  const int chunks = int(mx_ceil(K, kMxChunk));
  const int last = int(K - int64_t(chunks - 1) * kMxChunk) / 8;  // lanes of the last chunk
  // this warp's chunks: first, first + step, ...
  const int first = WPR == kMxWarps ? blockIdx.y * kMxWarps + warp : blockIdx.y;
  const int step = int(gridDim.y) * WPR;
  auto inside = [&](int c) { return c < chunks - 1 || (c == chunks - 1 && lane < last); };
  auto load = [&](int c) {
    return load_raw8<DT>(xr, int64_t(c) * kMxChunk);
  };

  float g = 1.f, g_inv = 1.f;
  if (FMT == LUTQ_NVFP4 && src >= 0) {
    // the row's largest finite magnitude (gridDim.y is 1)
    uint32_t m = 0;
    for (int c = first; c < chunks; c += step * 2 * kMxBatch) {
      Raw8<DT> raw[2 * kMxBatch];
#pragma unroll
      for (int u = 0; u < 2 * kMxBatch; ++u) {
        raw[u] = Raw8<DT>{};
        if (inside(c + u * step)) raw[u] = load(c + u * step);
      }
      uint32_t b[2 * kMxBatch], most = 0;
#pragma unroll
      for (int u = 0; u < 2 * kMxBatch; ++u) {
        b[u] = max_raw8<DT>(raw[u]);
        most = max(most, b[u]);
      }
      if (most >= raw_inf<DT>()) {  // leave out what is not finite
        most = 0;
#pragma unroll
        for (int u = 0; u < 2 * kMxBatch; ++u) {
          m = max(m, finite_max8<DT>(raw[u]));
        }
      }
      m = max(m, max_bits_f32<DT>(most));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (WPR == kMxWarps) {
      if (lane == 0) row_max[warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kMxWarps; ++w) m = max(m, row_max[w]);
    }
    g = nv_row_scale(m);
    g_inv = nv_row_scale_inverse(g);
  }
  bool bad = false;
  constexpr int L = FMT == LUTQ_MXFP4 ? 4 : 2;  // lanes per block
  uint8_t* codes = pm + lane * 4;
  uint8_t* scales = pm + mx_scale_off(rows, K) + (lane / (4 * L)) * 512;
  auto code_row = [&](int64_t r) { return codes + r * (K / 2); };
  auto scale_row = [&](int64_t r) {
    return scales + (r / kMxRowTile) * chunks * mx_chunk_bytes(FMT) + mx_scale_slot(r);
  };
  uint8_t* own_codes = code_row(item);
  uint8_t* own_scales = scale_row(item);
  for (int c = first; c < chunks; c += step * kMxBatch) {
    Raw8<DT> raw[kMxBatch];
#pragma unroll
    for (int u = 0; u < kMxBatch; ++u) {
      raw[u] = Raw8<DT>{};
      if (src >= 0 && inside(c + u * step)) raw[u] = load(c + u * step);
    }
    uint32_t q[kMxBatch], w[kMxBatch];
#pragma unroll
    for (int u = 0; u < kMxBatch; ++u) {
      // (zeros behind the row's end have the scale byte of zeros: 0)
      q[u] = w[u] = 0u;
      if (src >= 0 && c + u * step < chunks)
        q[u] = mx_quantize_lane<FMT, DT>(raw[u], g, g_inv, lane, &w[u], &bad);
    }
    auto store = [&](uint8_t* cr, uint8_t* sr) {
#pragma unroll
      for (int u = 0; u < kMxBatch; ++u) {
        const int cu = c + u * step;
        if (src >= 0 && inside(cu))
          *reinterpret_cast<uint32_t*>(cr + int64_t(cu) * (kMxChunk / 2)) = q[u];
        if ((lane & (4 * L - 1)) == 0 && cu < chunks)
          *reinterpret_cast<uint32_t*>(sr + int64_t(cu) * mx_chunk_bytes(FMT)) = w[u];
      }
    };
    if (!LISTED) {
      store(own_codes, own_scales);
    } else {
#pragma unroll 1
      for (int i = 0; i < copies; ++i) {
        const int r = i < 32 ? __shfl_sync(0xffffffffu, to_lane, i) : to[item * copies + i];
        if (r >= 0) store(code_row(r), scale_row(r));
      }
    }
  }
  if (FMT == LUTQ_NVFP4 && src >= 0 && (WPR == 1 || warp == 0) && lane == 0) {
    float* row_scales = reinterpret_cast<float*>(pm + mx_row_off(rows, K, FMT));
    for (int i = 0; i < (LISTED ? copies : 1); ++i) {
      const int64_t r = LISTED ? to[item * copies + i] : item;
      if (r >= 0) row_scales[r] = g;
    }
  }
  if (bad) report(dev_status, LUTQ_ERR_NONFINITE);
}

// nvfp4, many rows of up to 8192 values: a block takes a row at a time, holds
// it in registers between the search for its maximum and the rounding, and
// loads the next row meanwhile, so that every value is read once.
template <int DT>
__global__ void __launch_bounds__(kMxWarps * 32)
    mx_quantize_rows_kernel(const void* __restrict__ x, int64_t rows, int64_t K,
                            uint8_t* __restrict__ packed, int32_t* dev_status) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t row_max[2][kMxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int64_t esize = DT == LUTQ_FP32 ? 4 : 2;
  const int chunks = int(mx_ceil(K, kMxChunk));
  const int64_t padded = mx_ceil(rows, kMxRowTile) * kMxRowTile;
  const uint8_t* xl = static_cast<const uint8_t*>(x) + lane * 8 * esize;
  uint8_t* codes = packed + lane * 4;
  uint8_t* scales = packed + mx_scale_off(rows, K) + (lane / 8) * 512;
  float* row_scales = reinterpret_cast<float*>(packed + mx_row_off(rows, K, LUTQ_NVFP4));
  bool inside[kMxBatch];
#pragma unroll
  for (int u = 0; u < kMxBatch; ++u)
    inside[u] = int64_t(warp + u * kMxWarps) * kMxChunk + lane * 8 < K;
  auto load = [&](int64_t r, Raw8<DT> (&raw)[kMxBatch]) {
#pragma unroll
    for (int u = 0; u < kMxBatch; ++u) {
      raw[u] = Raw8<DT>{};
      if (r < rows && inside[u])
        raw[u] = load_raw8<DT>(xl + r * K * esize, int64_t(warp + u * kMxWarps) * kMxChunk);
    }
  };
  // rows in the order of their scales in the layout: the blocks that run at
  // the same time write neighbouring words (row i's tile, then i mod 32 of
  // its quarter (i / 32) mod 4)
  auto row_of = [&](int64_t i) {
    return i / kMxRowTile * kMxRowTile + (i & 3) * 32 + ((i & (kMxRowTile - 1)) >> 2);
  };
  bool bad = false;
  Raw8<DT> next[kMxBatch];
  if (blockIdx.x < padded) load(row_of(blockIdx.x), next);
  int flip = 0;
  for (int64_t i = blockIdx.x; i < padded; i += gridDim.x, flip ^= 1) {
    const int64_t r = row_of(i);
    Raw8<DT> raw[kMxBatch];
#pragma unroll
    for (int u = 0; u < kMxBatch; ++u) raw[u] = next[u];
    if (i + gridDim.x < padded) load(row_of(i + gridDim.x), next);
    uint32_t most = 0, m = 0;
#pragma unroll
    for (int u = 0; u < kMxBatch; ++u) most = max(most, max_raw8<DT>(raw[u]));
    if (most >= raw_inf<DT>()) {  // leave out what is not finite
      most = 0;
#pragma unroll
      for (int u = 0; u < kMxBatch; ++u) m = max(m, finite_max8<DT>(raw[u]));
    }
    m = __reduce_max_sync(0xffffffffu, max(m, max_bits_f32<DT>(most)));
    if (lane == 0) row_max[flip][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMxWarps; ++w) m = max(m, row_max[flip][w]);
    const float g = nv_row_scale(m), g_inv = nv_row_scale_inverse(g);
    uint8_t* cr = codes + r * (K / 2);
    uint8_t* sr =
        scales + (r / kMxRowTile) * chunks * mx_chunk_bytes(LUTQ_NVFP4) + mx_scale_slot(r);
#pragma unroll
    for (int u = 0; u < kMxBatch; ++u) {
      const int c = warp + u * kMxWarps;
      if (c >= chunks) break;
      uint32_t w;
      const uint32_t q = mx_quantize_lane<LUTQ_NVFP4, DT>(raw[u], g, g_inv, lane, &w, &bad);
      if (r < rows && inside[u]) *reinterpret_cast<uint32_t*>(cr + c * (kMxChunk / 2)) = q;
      if ((lane & 7) == 0)
        *reinterpret_cast<uint32_t*>(sr + int64_t(c) * mx_chunk_bytes(LUTQ_NVFP4)) = w;
    }
    if (threadIdx.x == 0 && r < rows) row_scales[r] = g;
  }
  if (bad) report(dev_status, LUTQ_ERR_NONFINITE);
}

// a * b cut toward zero, with the last bit set if anything was cut off: rounded
// to 16 bits from there, the exact product is rounded once.
__device__ __forceinline__ float mul_odd(float a, float b) {
  const float p = __fmul_rz(a, b), rest = fmaf(a, b, -p);
  return rest < 0.f || rest > 0.f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}

// The values of 8 codes: (element * scale) * row scale, rounded once.  The first
// product has 6 bits at most; the second is exact in fp32 if the row scale is a
// power of two (as the quantizer's are), and may have 30 bits otherwise.
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
  constexpr int L = FMT == LUTQ_MXFP4 ? 4 : 2;
  const uint8_t* codes = pm + r * (K / 2) + lane * 4;
  const uint8_t* sc = pm + mx_scale_off(rows, K) +
                      (r / kMxRowTile) * chunks * mx_chunk_bytes(FMT) + mx_scale_slot(r) +
                      (lane / (4 * L)) * 512 + ((lane / L) & 3);
  float g = 1.f;
  if (FMT == LUTQ_NVFP4) g = reinterpret_cast<const float*>(pm + mx_row_off(rows, K, FMT))[r];
  const bool odd = FMT == LUTQ_NVFP4 && DT != LUTQ_FP32 && (__float_as_uint(g) & 0x7fffffu) != 0u;
  const int64_t base = (int64_t(blockIdx.z) * rows + r) * K;
  constexpr int U = 2 * kMxBatch;
  for (int64_t c = blockIdx.y; c < chunks; c += int64_t(gridDim.y) * U) {
    uint32_t q[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t cu = c + u * int64_t(gridDim.y);
      q[u] = b[u] = 0;
      if (cu * kMxChunk + lane * 8 < K) {
        q[u] = *reinterpret_cast<const uint32_t*>(codes + cu * (kMxChunk / 2));
        b[u] = sc[cu * mx_chunk_bytes(FMT)];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = (c + u * int64_t(gridDim.y)) * kMxChunk + lane * 8;
      if (k >= K) break;
      const float s = FMT == LUTQ_MXFP4 ? e8m0_value(b[u]) : e4m3_value(b[u]);
      float v[8];
      e2m1_values8(q[u], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s;
      if (odd) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = mul_odd(v[j], g);
      } else if (FMT == LUTQ_NVFP4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= g;
      }
      store8<DT>(out, base + k, v);
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
      if (FMT == LUTQ_NVFP4) w &= 0x7f7f7f7fu;  // magnitudes: the tensor core's scales are unsigned
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

template <int FMT, int DT, bool LISTED>
static cudaError_t launch_quantize_l(const void* x, int64_t batch, int64_t items, int64_t rows,
                                     int64_t K, const int32_t* from, const int32_t* to,
                                     int copies, void* packed, int32_t* dev_status, int num_sms,
                                     cudaStream_t stream) {
  // few rows (fewer warps than eight blocks an SM have): a block takes a row
  const bool shared_row = items <= int64_t(num_sms) * kMxWarps;
  const int64_t padded = LISTED ? items : mx_ceil(rows, kMxRowTile) * kMxRowTile;
  const int64_t xs = rows * K, ps = mx_bytes(rows, K, FMT);
  uint8_t* out = static_cast<uint8_t*>(packed);
  if (shared_row) {
    // mxfp4 blocks along K as well, until every warp has a chunk or two
    const int64_t chunks = mx_ceil(K, kMxChunk);
    const unsigned gy =
        FMT == LUTQ_MXFP4 ? unsigned(std::min<int64_t>(mx_ceil(chunks, 2 * kMxWarps), 65535)) : 1u;
    return launch_pdl(mx_quantize_kernel<FMT, DT, kMxWarps, LISTED>,
                      dim3(unsigned(padded), gy, unsigned(batch)), dim3(kMxWarps * 32), 0, stream,
                      x, items, rows, K, from, to, copies, out, xs, ps, dev_status);
  }
  if constexpr (FMT == LUTQ_NVFP4 && !LISTED && DT != LUTQ_FP32) {
    if (batch == 1 && K <= kMxWarps * kMxBatch * kMxChunk)
      return launch_pdl(mx_quantize_rows_kernel<DT>, dim3(unsigned(num_sms) * 6),
                        dim3(kMxWarps * 32), 0, stream, x, rows, K, out, dev_status);
  }
  return launch_pdl(mx_quantize_kernel<FMT, DT, 1, LISTED>,
                    dim3(unsigned(mx_ceil(padded, kMxWarps)), 1u, unsigned(batch)),
                    dim3(kMxWarps * 32), 0, stream, x, items, rows, K, from, to, copies, out, xs,
                    ps, dev_status);
}

template <int FMT, int DT>
static cudaError_t launch_quantize_t(const void* x, int64_t batch, int64_t items, int64_t rows,
                                     int64_t K, const int32_t* from, const int32_t* to,
                                     int copies, void* packed, int32_t* dev_status, int num_sms,
                                     cudaStream_t stream) {
  return to != nullptr ? launch_quantize_l<FMT, DT, true>(x, batch, items, rows, K, from, to,
                                                          copies, packed, dev_status, num_sms,
                                                          stream)
                       : launch_quantize_l<FMT, DT, false>(x, batch, items, rows, K, from, to,
                                                           copies, packed, dev_status, num_sms,
                                                           stream);
}

// `items` source rows into a packed buffer of `rows` rows (see the kernel).
cudaError_t launch_mx_quantize(const void* x, int dtype, int64_t batch, int64_t items,
                               int64_t rows, int64_t K, int fmt, const int32_t* from,
                               const int32_t* to, int copies, void* packed, int32_t* dev_status,
                               int num_sms, cudaStream_t stream) {
  auto go = [&](auto f) {
    return f(x, batch, items, rows, K, from, to, copies, packed, dev_status, num_sms, stream);
  };
  if (fmt == LUTQ_MXFP4) {
    if (dtype == LUTQ_BF16) return go(launch_quantize_t<LUTQ_MXFP4, LUTQ_BF16>);
    if (dtype == LUTQ_FP16) return go(launch_quantize_t<LUTQ_MXFP4, LUTQ_FP16>);
    return go(launch_quantize_t<LUTQ_MXFP4, LUTQ_FP32>);
  }
  if (dtype == LUTQ_BF16) return go(launch_quantize_t<LUTQ_NVFP4, LUTQ_BF16>);
  if (dtype == LUTQ_FP16) return go(launch_quantize_t<LUTQ_NVFP4, LUTQ_FP16>);
  return go(launch_quantize_t<LUTQ_NVFP4, LUTQ_FP32>);
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
