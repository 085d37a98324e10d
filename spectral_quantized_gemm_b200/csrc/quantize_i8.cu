// 8-bit integer quantization of a matrix with one scale for each row and / or each column.
//
// For a line (a row, or a column for the transposed output) with amax = max |x| over its
// finite entries:
//   a = max(amax, 127 * 2^-126),  scale = RN(a / 127),  code = rint(127 x / a),
// the quotient exact and ties to even; NaN gives 0 and an infinity +-127 (both raise
// METIS_DEV_NONFINITE).  The floor on a keeps the scale a normal number, also for a line
// of zeros.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace metis {
namespace {

constexpr float kMinAmax = 127.0f * 1.17549435e-38f;   // 127 * 2^-126, exact

// |x| of a finite value as its fp32 bits (they order like the values), else 0.
__device__ __forceinline__ uint32_t finite_abs_bits(float x, bool& nonfinite) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  if (b >= 0x7F800000u) {
    nonfinite = true;
    return 0u;
  }
  return b;
}

struct LineScale {
  float a;     // max(amax, kMinAmax)
  float inv;   // RN(127 / a)
};

__device__ __forceinline__ LineScale line_scale(uint32_t amax_bits) {
  LineScale s;
  s.a = fmaxf(__uint_as_float(amax_bits), kMinAmax);
  s.inv = __fdiv_rn(127.0f, s.a);
  return s;
}

// rint(127 x / a).  x * inv is within 127 * 2^-23 < 2^-16 of the quotient, which decides the
// code unless the quotient lies that close to a border half way between two integers; there
// the two sides of 127 |x| <> (q + 1/2) a are compared, both exact in fp64 (24 + 8 bits).
__device__ __forceinline__ int code_i8(float x, const LineScale& s) {
  const float y = fminf(fabsf(x) * s.inv, 127.0f);   // an infinity saturates
  const float q = floorf(y);
  const float frac = y - q;
  int c;
  if (fabsf(frac - 0.5f) >= 6.1035156e-5f) {         // 2^-14
    c = (int)q + (frac > 0.5f ? 1 : 0);
  } else {
    const double l = 254.0 * (double)fabsf(x), r = (2.0 * (double)q + 1.0) * (double)s.a;
    c = (int)q + (l > r || (l == r && ((int)q & 1)) ? 1 : 0);
  }
  if (!(x == x)) c = 0;                              // fminf drops a NaN
  return x < 0.0f ? -c : c;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

// Eight consecutive elements of a row from column c on; columns >= cols read as 0.
// `vec`: the row start is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t c, int64_t cols, bool vec, float (&x)[8]) {
  if (vec && c + 8 <= cols) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4*>(row + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
      const float4 u = *reinterpret_cast<const float4*>(row + c);
      const float4 v = *reinterpret_cast<const float4*>(row + c + 4);
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
      x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = c + i < cols ? to_f32<T>(row[c + i]) : 0.0f;
  }
}

// Eight codes packed into 8 bytes; the bytes of columns >= cols are not written.
__device__ __forceinline__ void store8(int8_t* row, int64_t c, int64_t cols, const int (&q)[8]) {
  if (c + 8 <= cols) {
    uint2 w;
    w.x = (uint32_t)(q[0] & 255) | ((uint32_t)(q[1] & 255) << 8) | ((uint32_t)(q[2] & 255) << 16) | ((uint32_t)q[3] << 24);
    w.y = (uint32_t)(q[4] & 255) | ((uint32_t)(q[5] & 255) << 8) | ((uint32_t)(q[6] & 255) << 16) | ((uint32_t)q[7] << 24);
    *reinterpret_cast<uint2*>(row + c) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = (int8_t)q[i];
  }
}

// One row per block: maximum, then codes.
template <typename T>
__global__ void __launch_bounds__(256) quantize_i8_rows_kernel(const T* __restrict__ M, int64_t rows, int64_t cols,
                                                               int64_t ld, int8_t* __restrict__ codes, int64_t ldq,
                                                               float* __restrict__ scales, uint32_t* status) {
  __shared__ uint32_t part[8];
  tc::grid_launch_dependents();   // a product that follows may start loading its other operand
  const int64_t r = blockIdx.x;
  const T* row = M + r * ld;
  const bool vec = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
  uint32_t top = 0;
  bool bad = false;
  for (int64_t c = (int64_t)threadIdx.x * 8; c < cols; c += 256 * 8) {
    float x[8];
    load8(row, c, cols, vec, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, finite_abs_bits(x[i], bad));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, part[i]);
  const LineScale s = line_scale(top);
  if (threadIdx.x == 0) scales[r] = __fdiv_rn(s.a, 127.0f);
  if (bad) raise_status(status, METIS_DEV_NONFINITE);
  for (int64_t c = (int64_t)threadIdx.x * 8; c < cols; c += 256 * 8) {
    float x[8];
    int q[8];
    load8(row, c, cols, vec, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = code_i8(x[i], s);
    store8(codes + r * ldq, c, cols, q);
  }
}

// Maxima of rows (row_top, nullable) and columns of a 64 x 256 tile, joined by integer
// atomicMax on the bits of |x| (the result does not depend on the order).
constexpr int kTopRows = 64, kTopCols = 256;
template <typename T>
__global__ void __launch_bounds__(256) line_tops_kernel(const T* __restrict__ M, int64_t rows, int64_t cols, int64_t ld,
                                                        uint32_t* row_top, uint32_t* col_top, uint32_t* status) {
  __shared__ uint32_t part[8][kTopCols + 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tiles_c = (cols + kTopCols - 1) / kTopCols;
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * kTopRows, c0 = (int64_t)(blockIdx.x % tiles_c) * kTopCols;
  uint32_t top[8] = {};
  bool bad = false;
#pragma unroll 4
  for (int i = 0; i < kTopRows / 8; ++i) {
    const int64_t r = r0 + i * 8 + warp;
    uint32_t rt = 0;
    if (r < rows) {
      const T* row = M + r * ld;
      float x[8];
      load8(row, c0 + lane * 8, cols, (reinterpret_cast<uintptr_t>(row) & 15u) == 0, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b = finite_abs_bits(x[j], bad);
        top[j] = max(top[j], b);
        rt = max(rt, b);
      }
    }
    if (row_top) {
      rt = __reduce_max_sync(0xffffffffu, rt);
      if (lane == 0 && rt) atomicMax(&row_top[r], rt);
    }
  }
  if (bad) raise_status(status, METIS_DEV_NONFINITE);
#pragma unroll
  for (int j = 0; j < 8; ++j) part[warp][lane * 8 + j] = top[j];
  __syncthreads();
  uint32_t t = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) t = max(t, part[w][threadIdx.x]);
  const int64_t c = c0 + threadIdx.x;
  if (c < cols && t) atomicMax(&col_top[c], t);
}

// Codes of a 128 x 64 tile from the maxima: row-wise (codes_r nullable) straight from the
// registers, column-wise through shared memory so that each column leaves as 128 bytes.
constexpr int kTileRows = 128, kTileCols = 64;
template <typename T>
__global__ void __launch_bounds__(256) quantize_i8_tiles_kernel(const T* __restrict__ M, int64_t rows, int64_t cols,
                                                                int64_t ld, const uint32_t* __restrict__ row_top,
                                                                const uint32_t* __restrict__ col_top,
                                                                int8_t* __restrict__ codes_r, int64_t ldr,
                                                                int8_t* __restrict__ codes_c, int64_t ldc) {
  __shared__ uint32_t tile[kTileCols][kTileRows / 4 + 1];   // four rows of a column in each word
  const int64_t tiles_c = (cols + kTileCols - 1) / kTileCols;
  const int64_t r0 = (int64_t)(blockIdx.x / tiles_c) * kTileRows, c0 = (int64_t)(blockIdx.x % tiles_c) * kTileCols;
  const int chunk = threadIdx.x & 7, group = threadIdx.x >> 3;   // 8 columns, 4 rows
  const int64_t c = c0 + chunk * 8;
  LineScale cs[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cs[j] = line_scale(c + j < cols ? col_top[c + j] : 0u);
  uint32_t packed[8] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + group * 4 + i;
    if (r >= rows || c >= cols) continue;
    const T* row = M + r * ld;
    float x[8];
    load8(row, c, cols, (reinterpret_cast<uintptr_t>(row) & 15u) == 0, x);
    if (codes_r) {
      const LineScale s = line_scale(row_top[r]);
      int q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = code_i8(x[j], s);
      store8(codes_r + r * ldr, c, cols, q);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) packed[j] |= (uint32_t)(code_i8(x[j], cs[j]) & 255) << (8 * i);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) tile[chunk * 8 + j][group] = packed[j];
  __syncthreads();
  // 16 rows (16 bytes) of a column per thread and step
#pragma unroll
  for (int u = threadIdx.x; u < kTileCols * 8; u += 256) {
    const int64_t cc = c0 + (u >> 3), rr = r0 + (u & 7) * 16;
    if (cc >= cols || rr >= rows) continue;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = tile[u >> 3][(u & 7) * 4 + i];
    int8_t* dst = codes_c + cc * ldc + rr;
    if (rr + 16 <= rows) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (rr + i < rows) dst[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
  }
}

// Zeroes, or turns maxima into scales in place.
__global__ void zero_tops_kernel(uint32_t* a, int64_t na, uint32_t* b, int64_t nb) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < na) a[i] = 0;
  if (i >= na && i - na < nb) b[i - na] = 0;
}
__global__ void tops_to_scales_kernel(float* a, int64_t na, float* b, int64_t nb) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  float* s = i < na ? a + i : (i - na < nb ? b + (i - na) : nullptr);
  if (s) *s = __fdiv_rn(fmaxf(*s, kMinAmax), 127.0f);
}

template <typename T>
cudaError_t run_quantize(const T* M, int64_t rows, int64_t cols, int64_t ld, const metis_int8* row,
                         const metis_int8* col, uint32_t* status, cudaStream_t st) {
  if (!col) {
    quantize_i8_rows_kernel<T><<<(unsigned)rows, 256, 0, st>>>(M, rows, cols, ld, row->codes, row->ld, row->scales, status);
    count_launch();
    return cudaGetLastError();
  }
  // The maxima are gathered in the scale arrays themselves and turned into scales last.
  uint32_t* row_top = row ? reinterpret_cast<uint32_t*>(row->scales) : nullptr;
  uint32_t* col_top = reinterpret_cast<uint32_t*>(col->scales);
  const int64_t nr = row ? rows : 0;
  const unsigned lines = (unsigned)((nr + cols + 255) / 256);
  zero_tops_kernel<<<lines, 256, 0, st>>>(row_top, nr, col_top, cols);
  const int64_t tops = ((rows + kTopRows - 1) / kTopRows) * ((cols + kTopCols - 1) / kTopCols);
  line_tops_kernel<T><<<(unsigned)tops, 256, 0, st>>>(M, rows, cols, ld, row_top, col_top, status);
  const int64_t tiles = ((rows + kTileRows - 1) / kTileRows) * ((cols + kTileCols - 1) / kTileCols);
  quantize_i8_tiles_kernel<T><<<(unsigned)tiles, 256, 0, st>>>(M, rows, cols, ld, row_top, col_top,
                                                               row ? row->codes : nullptr, row ? row->ld : 0,
                                                               col->codes, col->ld);
  tops_to_scales_kernel<<<lines, 256, 0, st>>>(row ? row->scales : nullptr, nr, col->scales, cols);
  count_launch(4);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_i8(const void* M, bool bf16, int64_t rows, int64_t cols, int64_t ld, const metis_int8* row,
                               const metis_int8* col, uint32_t* status, cudaStream_t st) {
  if (bf16)
    return run_quantize(static_cast<const __nv_bfloat16*>(M), rows, cols, ld, row, col, status, st);
  return run_quantize(static_cast<const float*>(M), rows, cols, ld, row, col, status, st);
}

}  // namespace metis
