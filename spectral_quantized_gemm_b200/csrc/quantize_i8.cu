// 8-bit integer quantization of a matrix with one scale for each row and / or each column.
//
// For a line (a row, or a column for the transposed output) with amax = max |x| over its
// finite entries:
//   a = max(amax, 127 * 2^-126),  scale = RN(a / 127),  code = rint(127 x / a),
// the quotient exact and ties to even; NaN gives 0 and an infinity +-127 (both raise
// METIS_DEV_NONFINITE).  The floor on a keeps the scale a normal number, also for a line
// of zeros.
//
// The quotient.  127 / a is held in two fp32 words, inv + lo (lo is the rounded remainder of
// the rounded quotient over a, so their sum is off by 2^-46 of it), and
//   y = fma(x, inv, x lo)
// is the fp32 number nearest to 127 x / a, up to 2^-24 of an ulp.  Adding 1.5 * 2^23 rounds
// it to an integer, ties to even, in the low byte.
//   bf16 x: a quotient half way between two integers is itself an fp32 number, so y is that
//     number; every other quotient of two 8-bit mantissas differs from such a border by
//     2^-16 of itself or more (254 X - (2 n + 1) A is an integer), y by 2^-24.  y decides.
//   fp32 x: where y lies within 2^-15 of a border, the two sides of 254 |x| <> (2 n + 1) a
//     are compared in fp64, both exact (24 + 8 bits).  One element in 2^14.
// Lines with a > 2^100 (lo would be subnormal) or with entries that are not finite take the
// fp64 comparison for every element.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace metis {
namespace {

constexpr float kMinAmax = 127.0f * 1.17549435e-38f;   // 127 * 2^-126, exact
constexpr uint32_t kInf = 0x7F800000u;
constexpr int kThreads = 256;

struct LineScale {
  float a;         // max(amax, kMinAmax); its sign says that every element needs the comparison
  float inv, lo;   // 127 / a
};

__device__ __forceinline__ LineScale line_scale(uint32_t amax_bits, bool nonfinite) {
  LineScale s;
  const float a = fmaxf(__uint_as_float(amax_bits), kMinAmax);
  s.inv = __fdiv_rn(127.0f, a);
  s.lo = __fdiv_rn(__fmaf_rn(-s.inv, a, 127.0f), a);
  s.a = nonfinite || a > 1.2676506e30f ? -a : a;       // 2^100
  return s;
}
__device__ __forceinline__ float scale_of(const LineScale& s) { return __fdiv_rn(fabsf(s.a), 127.0f); }

// The code by exact comparison, for any x.
__device__ __noinline__ int code_exact(float x, float a, float inv) {
  if (!(x == x)) return 0;
  const double m = fmin(fabs((double)x), (double)a);   // an infinity saturates
  const float y = fminf((float)m * inv, 127.0f);       // within 2^-16 of the quotient
  // the code is the number of borders (n + 1/2) below the quotient; y finds the nearest one
  const int n = (int)floorf(y);                         // the border n + 1/2, or one of its neighbours
  int c = max(n - 1, 0);
  for (int k = c; k <= n + 1 && k < 127; ++k) {
    const double l = 254.0 * m, r = (2.0 * k + 1.0) * (double)a;
    if (l > r || (l == r && (k & 1))) c = k + 1;
  }
  return x < 0.0f ? -c : c;
}

template <typename T>
__device__ __forceinline__ uint32_t code_bits(float x, const LineScale& s, bool& near) {
  const float y = __fmaf_rn(x, s.inv, __fmul_rn(x, s.lo));
  const float t = __fadd_rn(y, 12582912.0f);
  if (sizeof(T) == 4) near |= fabsf(__fsub_rn(y, __fsub_rn(t, 12582912.0f))) > 0.49996f;
  return __float_as_uint(t);
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Eight consecutive elements of a row as they are in memory.
template <typename T>
struct Chunk {
  uint32_t w[2 * sizeof(T)];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
};

// Elements from column c on; columns >= cols read as 0.  vec: the row starts on 16 bytes.
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int64_t c, int64_t cols, bool vec) {
  Chunk<T> k;
  if (vec && c + 8 <= cols) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(row + c)[i];
      k.w[4 * i] = u.x; k.w[4 * i + 1] = u.y; k.w[4 * i + 2] = u.z; k.w[4 * i + 3] = u.w;
    }
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) k.w[i] = c + i < cols ? reinterpret_cast<const uint32_t*>(row)[c + i] : 0u;
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      k.w[i] = (c + 2 * i < cols ? (uint32_t)h[c + 2 * i] : 0u) | (c + 2 * i + 1 < cols ? (uint32_t)h[c + 2 * i + 1] << 16 : 0u);
  }
  return k;
}

// Largest |x| as fp32 bits (they order like the values); NaN and infinities give kInf or more.
template <typename T>
__device__ __forceinline__ uint32_t chunk_top(const Chunk<T>& k, uint32_t top) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, k.w[i] & 0x7FFFFFFFu);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, k.w[i] & 0x7FFF7FFFu);
    top = max(top, max(m << 16, m & 0xFFFF0000u));
  }
  return top;
}
// The same over finite entries only.
template <typename T>
__device__ __forceinline__ uint32_t chunk_finite_top(const Chunk<T>& k, uint32_t top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(k.get(i)) & 0x7FFFFFFFu;
    if (b < kInf) top = max(top, b);
  }
  return top;
}

// The eight codes of a chunk under one scale, packed.
template <typename T>
__device__ __noinline__ uint2 chunk_codes_exact(Chunk<T> k, float a, float inv) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = (uint32_t)code_exact(k.get(i), a, inv);
  return make_uint2(pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]));
}
__device__ __noinline__ uint32_t four_codes_exact(float x0, float x1, float x2, float x3, float a, float inv) {
  return pack4((uint32_t)code_exact(x0, a, inv), (uint32_t)code_exact(x1, a, inv), (uint32_t)code_exact(x2, a, inv),
               (uint32_t)code_exact(x3, a, inv));
}
template <typename T>
__device__ __forceinline__ uint2 chunk_codes(const Chunk<T>& k, const LineScale& s) {
  uint32_t b[8];
  bool near = s.a < 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = code_bits<T>(k.get(i), s, near);
  if (near) return chunk_codes_exact(k, fabsf(s.a), s.inv);
  return make_uint2(pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]));
}

// Eight codes; the bytes of columns >= cols are not written.
__device__ __forceinline__ void store_codes(int8_t* row, int64_t c, int64_t cols, uint2 w) {
  if (c + 8 <= cols) {
    *reinterpret_cast<uint2*>(row + c) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = (int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}

// ---------------------------------------------------------------- rows
// GROUP threads take a row and hold it, four chunks each at most, between the maximum and the
// codes, so it is read once.  HELD false: a row too long for that is read again, from L2.
// (A warp a row with 16 chunks each took 128 registers, a quarter of the SM's warps, and 27 us at
// 8192 x 4096 bf16.)
constexpr int kHeld = 4;

template <typename T, int GROUP, bool HELD>
__global__ void __launch_bounds__(GROUP > kThreads ? GROUP : kThreads)
    quantize_i8_rows_kernel(const T* __restrict__ M, int64_t rows, int64_t cols, int64_t ld, int8_t* __restrict__ codes,
                            int64_t ldq, float* __restrict__ scales, uint32_t* status) {
  constexpr int BLOCK = GROUP > kThreads ? GROUP : kThreads;
  __shared__ uint32_t part[2][BLOCK / 32];
  tc::grid_launch_dependents();   // a product that follows may start loading its other operand
  const int t = threadIdx.x % GROUP;
  const int64_t r = (int64_t)blockIdx.x * (BLOCK / GROUP) + threadIdx.x / GROUP;
  const T* row = M + min(r, rows - 1) * ld;   // a group past the last row repeats it and writes nothing
  int8_t* out = codes + r * ldq;
  const bool vec = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;

  auto over_row = [&](uint32_t top, int slot) {
    top = __reduce_max_sync(0xffffffffu, top);
    if (GROUP > 32) {
      if ((threadIdx.x & 31) == 0) part[slot][threadIdx.x >> 5] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < GROUP / 32; ++i) top = max(top, part[slot][(threadIdx.x / GROUP) * (GROUP / 32) + i]);
    }
    return top;
  };

  uint32_t top = 0;
  Chunk<T> held[kHeld];
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = load_chunk(row, (int64_t)(i * GROUP + t) * 8, cols, vec);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) top = chunk_top(held[i], top);
  } else {
    for (int64_t c = (int64_t)t * 8; c < cols; c += GROUP * 8) top = chunk_top(load_chunk(row, c, cols, vec), top);
  }
  top = over_row(top, 0);
  const bool bad = top >= kInf;
  if (__syncthreads_or(bad)) {
    uint32_t fine = 0;
    for (int64_t c = (int64_t)t * 8; c < cols; c += GROUP * 8) fine = chunk_finite_top(load_chunk(row, c, cols, vec), fine);
    fine = over_row(fine, 1);
    if (bad) top = fine;
  }
  if (r >= rows) return;
  const LineScale s = line_scale(top, bad);
  if (t == 0) {
    scales[r] = scale_of(s);
    if (bad) raise_status(status, METIS_DEV_NONFINITE);
  }
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (int64_t)(i * GROUP + t) * 8;
      if (c < cols) store_codes(out, c, cols, chunk_codes(held[i], s));
    }
  } else {
    for (int64_t c = (int64_t)t * 8; c < cols; c += GROUP * 8)
      store_codes(out, c, cols, chunk_codes(load_chunk(row, c, cols, vec), s));
  }
}

// ---------------------------------------------------------------- columns
// A cluster takes a strip of 64 columns, each of its blocks a share of the rows: maxima of
// the share, joined through distributed shared memory, then the codes of the share in slabs
// of 128 rows, transposed through shared memory so that a column leaves as 128 bytes.  The
// second reading of a share finds it in L2 (the strips under way hold some 40 MB of its 126).
constexpr int kStrip = 64, kSlab = 128;

template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_i8_cols_kernel(const T* __restrict__ M, int64_t rows, int64_t cols,
                                                                    int64_t ld, int8_t* __restrict__ codes, int64_t ldq,
                                                                    float* __restrict__ scales, uint32_t* status) {
  __shared__ uint32_t part[kThreads / 32][kStrip];
  __shared__ uint32_t tops[2][kStrip];
  __shared__ LineScale line[kStrip];
  __shared__ uint32_t tile[2][kStrip][kSlab / 4 + 1];   // four rows of a column in each word
  const int share = (int)tc::cluster_rank(), shares = (int)tc::cluster_size();
  const int64_t c0 = (int64_t)(blockIdx.x / shares) * kStrip;
  const int64_t slabs = (rows + kSlab - 1) / kSlab;
  const int64_t first = slabs * share / shares, last = slabs * (share + 1) / shares;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunk = threadIdx.x & 7, group = threadIdx.x >> 3;   // 8 columns, 4 rows
  const int64_t c = c0 + chunk * 8;
  const bool vec = ((reinterpret_cast<uintptr_t>(M) | (uintptr_t)(ld * (int64_t)sizeof(T))) & 15u) == 0;
  auto load_slab = [&](int64_t s, Chunk<T> (&k)[4]) {
    const int64_t r0 = s * kSlab + group * 4;
    const T* at = M + r0 * ld;
    if (r0 + 4 <= rows) {
#pragma unroll
      for (int i = 0; i < 4; ++i, at += ld) k[i] = load_chunk(at, c, cols, vec);
    } else {   // the last row again does not change a maximum, and its codes are not written
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = load_chunk(M + min(r0 + i, rows - 1) * ld, c, cols, vec);
    }
  };

  // Maxima of the strip's columns over all rows, in shared memory of every block.
  auto column_tops = [&](bool finite_only, int slot) {
    uint32_t top[8] = {};
    if (sizeof(T) == 2 && !finite_only) {
      uint32_t two[4] = {};
      for (int64_t s = first; s < last; ++s) {
        Chunk<T> k[4];
        load_slab(s, k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) two[j] = __vmaxu2(two[j], k[i].w[j] & 0x7FFF7FFFu);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        top[2 * j] = two[j] << 16;
        top[2 * j + 1] = two[j] & 0xFFFF0000u;
      }
    } else {
      for (int64_t s = first; s < last; ++s) {
        Chunk<T> k[4];
        load_slab(s, k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t b = __float_as_uint(k[i].get(j)) & 0x7FFFFFFFu;
            if (!finite_only || b < kInf) top[j] = max(top[j], b);
          }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 8));
      top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
      if (lane < 8) part[warp][chunk * 8 + j] = top[j];
    }
    __syncthreads();
    if (threadIdx.x < kStrip) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) m = max(m, part[w][threadIdx.x]);
      tops[slot][threadIdx.x] = m;
    }
    tc::cluster_sync();
    uint32_t m = 0;
    if (threadIdx.x < kStrip) {
      const uint32_t at = tc::smem_addr(&tops[slot][threadIdx.x]);
      for (int s = 0; s < shares; ++s) m = max(m, tc::load_cluster_u32(tc::cluster_addr_u32(at, (uint32_t)s)));
    }
    return m;   // of column c0 + threadIdx.x, in the first 64 threads
  };

  uint32_t top = column_tops(false, 0);
  const bool bad = threadIdx.x < kStrip && top >= kInf;
  if (__syncthreads_or(bad)) {                 // the same in all blocks of the cluster
    const uint32_t fine = column_tops(true, 1);
    if (bad) top = fine;
  }
  if (threadIdx.x < kStrip) {
    const LineScale s = line_scale(top, bad);
    line[threadIdx.x] = s;
    if (share == 0 && c0 + threadIdx.x < cols) {
      scales[c0 + threadIdx.x] = scale_of(s);
      if (bad) raise_status(status, METIS_DEV_NONFINITE);
    }
  }
  tc::cluster_arrive();                        // this block has read the others' maxima
  __syncthreads();
  LineScale ls[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) ls[j] = line[chunk * 8 + j];

  int buf = 0;
  for (int64_t s = first; s < last; ++s, buf ^= 1) {
    const int64_t r0 = s * kSlab;
    Chunk<T> k[4];
    load_slab(s, k);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t b[4];
      bool near = ls[j].a < 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = code_bits<T>(k[i].get(j), ls[j], near);
      uint32_t w = pack4(b[0], b[1], b[2], b[3]);
      if (near) w = four_codes_exact(k[0].get(j), k[1].get(j), k[2].get(j), k[3].get(j), fabsf(ls[j].a), ls[j].inv);
      tile[buf][chunk * 8 + j][group] = w;
    }
    __syncthreads();   // the other buffer was read before the block came here
    // 16 rows (16 bytes) of a column per thread and step
#pragma unroll
    for (int u = threadIdx.x; u < kStrip * 8; u += kThreads) {
      const int64_t cc = c0 + (u >> 3), rr = r0 + (u & 7) * 16;
      if (cc >= cols || rr >= rows) continue;
      const uint32_t* from = &tile[buf][u >> 3][(u & 7) * 4];
      int8_t* dst = codes + cc * ldq + rr;
      if (rr + 16 <= rows) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(from[0], from[1], from[2], from[3]);
      } else {
        for (int i = 0; rr + i < rows; ++i) dst[i] = (int8_t)(from[i >> 2] >> (8 * (i & 3)));
      }
    }
  }
  tc::cluster_wait();                          // nor does a block leave while its own are read
  tc::grid_dependency_wait();                  // the row kernel before this one, beside which it ran
}

template <typename T, int GROUP, bool HELD>
cudaError_t launch_rows(const T* M, int64_t rows, int64_t cols, int64_t ld, const metis_int8* q, uint32_t* status,
                        cudaStream_t st) {
  constexpr int BLOCK = GROUP > kThreads ? GROUP : kThreads;
  const int64_t blocks = (rows + BLOCK / GROUP - 1) / (BLOCK / GROUP);
  quantize_i8_rows_kernel<T, GROUP, HELD><<<(unsigned)blocks, BLOCK, 0, st>>>(M, rows, cols, ld, q->codes, q->ld, q->scales, status);
  count_launch();
  return cudaGetLastError();
}

// The smallest group that holds a row; where rows are too few to fill the SMs, the largest that
// has a chunk for each thread.
template <typename T>
cudaError_t run_rows(const T* M, int64_t rows, int64_t cols, int64_t ld, const metis_int8* q, uint32_t* status, int sm_count,
                     cudaStream_t st) {
  const int64_t chunks = (cols + 7) / 8;
  if (chunks > 512 * kHeld) return launch_rows<T, 512, false>(M, rows, cols, ld, q, status, st);
  const bool few = rows < 4 * (int64_t)sm_count;
  if (few ? chunks <= 64 : chunks <= 32 * kHeld) return launch_rows<T, 32, true>(M, rows, cols, ld, q, status, st);
  if (few ? chunks <= 256 : chunks <= 128 * kHeld) return launch_rows<T, 128, true>(M, rows, cols, ld, q, status, st);
  return launch_rows<T, 512, true>(M, rows, cols, ld, q, status, st);
}

// beside: the launch before this one on the stream is the row kernel of the same matrix (an
// ordinary launch); the two run side by side.
template <typename T>
cudaError_t run_cols(const T* M, int64_t rows, int64_t cols, int64_t ld, const metis_int8* q, uint32_t* status, bool beside,
                     cudaStream_t st) {
  const int64_t slabs = (rows + kSlab - 1) / kSlab;
  const int shares = (int)std::min<int64_t>(8, slabs);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((cols + kStrip - 1) / kStrip * shares));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)shares;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, quantize_i8_cols_kernel<T>, M, rows, cols, ld, q->codes, q->ld, q->scales, status);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T>
cudaError_t run_quantize(const T* M, int64_t rows, int64_t cols, int64_t ld, const metis_int8* row, const metis_int8* col,
                         uint32_t* status, int sm_count, cudaStream_t st) {
  if (row) {
    const cudaError_t e = run_rows(M, rows, cols, ld, row, status, sm_count, st);
    if (e != cudaSuccess || !col) return e;
  }
  return run_cols(M, rows, cols, ld, col, status, row != nullptr, st);
}

}  // namespace

cudaError_t launch_quantize_i8(const void* M, bool bf16, int64_t rows, int64_t cols, int64_t ld, const metis_int8* row,
                               const metis_int8* col, uint32_t* status, int sm_count, cudaStream_t st) {
  if (bf16)
    return run_quantize(static_cast<const __nv_bfloat16*>(M), rows, cols, ld, row, col, status, sm_count, st);
  return run_quantize(static_cast<const float*>(M), rows, cols, ld, row, col, status, sm_count, st);
}

}  // namespace metis
