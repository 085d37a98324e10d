// 8-bit integer quantization of a matrix with one scale for each row and / or each column.
//
// For a line (a row, or a column for the transposed output) with amax = max |x| over its
// finite entries:
//   a = max(amax, 127 * 2^-126),  scale = RN(a / 127),  code = rint(127 x / a),
// the quotient exact and ties to even; NaN gives 0 and an infinity +-127 (both raise
// METIS_DEV_NONFINITE).  The floor on a keeps the scale a normal number, also for a line
// of zeros.
//
// The quotient.  127 / a is held in two fp32 words, inv from an approximate reciprocal r of a
// (2^-22) and lo = (127 - inv a) r, so their sum is off by 2^-44 of it, and
//   y = fma(x, inv, x lo)
// is the fp32 number nearest to 127 x / a, up to 2^-20 of an ulp.  Adding 1.5 * 2^23 rounds
// it to an integer, ties to even, in the low byte.
//   bf16 x: a quotient half way between two integers is itself an fp32 number, so y is that
//     number; every other quotient of two 8-bit mantissas differs from such a border by
//     2^-16 of itself or more (254 X - (2 n + 1) A is an integer), y by 2^-24.  y decides.
//   fp32 x: where y lies within 2^-15 of a border (one element in 2^14), the two sides of
//     254 |x| <> (2 n + 1) a are compared, each an fp32 product and its exact remainder.
// Lines whose a lies outside 2^-90 .. 2^100 (a remainder could be subnormal) or with entries
// that are not finite take a comparison in fp64 (24 + 8 bits: exact) for every element.
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
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(a));
  s.inv = __fmul_rn(127.0f, r);
  s.lo = __fmul_rn(__fmaf_rn(-s.inv, a, 127.0f), r);
  // 2^100 and 2^-90; a line of zeros needs no comparison
  s.a = nonfinite || a > 1.2676506e30f || (amax_bits != 0 && a < 8.0779357e-28f) ? -a : a;
  return s;
}
__device__ __forceinline__ float scale_of(const LineScale& s) { return __fdiv_rn(fabsf(s.a), 127.0f); }

// The code by exact comparison, for any x.
__device__ __noinline__ int code_exact(float x, float a, float inv) {
  if (!(x == x)) return 0;
  const double m = fmin(fabs((double)x), (double)a);   // an infinity saturates
  const float y = fminf((float)m * inv, 127.0f);       // within 2^-14 of the quotient
  // the code is the number of borders (n + 1/2) below the quotient; y finds the nearest one
  const int n = (int)floorf(y);                         // the border n + 1/2, or one of its neighbours
  int c = max(n - 1, 0);
  for (int k = c; k <= n + 1 && k < 127; ++k) {
    const double l = 254.0 * m, r = (2.0 * k + 1.0) * (double)a;
    if (l > r || (l == r && (k & 1))) c = k + 1;
  }
  return x < 0.0f ? -c : c;
}

// The codes of two elements in the low bytes, for a line that needs no fp64 comparison; fp32: `border`
// becomes the largest distance from an integer, near a half the code is open.
template <typename T>
__device__ __forceinline__ void code_bits(float x0, float x1, const LineScale& s, uint32_t& b0, uint32_t& b1, float& border) {
  const Pair x(x0, x1), magic(12582912.0f);
  const Pair y = fma2(x, Pair(s.inv), x * Pair(s.lo)), t = y + magic;
  float t0, t1;
  t.get(t0, t1);
  b0 = __float_as_uint(t0);
  b1 = __float_as_uint(t1);
  if constexpr (sizeof(T) == 4) {
    float d0, d1;
    fma2(t + Pair(-12582912.0f), Pair(-1.0f), y).get(d0, d1);
    border = fmaxf(border, fmaxf(fabsf(d0), fabsf(d1)));
  }
}
// The code of one element with the comparison.
__device__ __forceinline__ uint32_t code_at_border(float x, const LineScale& s) {
  const float y = __fmaf_rn(x, s.inv, __fmul_rn(x, s.lo));
  const float t = __fadd_rn(y, 12582912.0f);
  if (!(fabsf(__fsub_rn(y, __fsub_rn(t, 12582912.0f))) > 0.49996f)) return __float_as_uint(t);
  const float m = fabsf(x), n = floorf(fabsf(y)), odd = 2.0f * n + 1.0f;
  const float l = __fmul_rn(254.0f, m), r = __fmul_rn(odd, s.a);
  const float d = __fadd_rn(__fsub_rn(l, r), __fsub_rn(__fmaf_rn(254.0f, m, -l), __fmaf_rn(odd, s.a, -r)));
  const float c = n + (d > 0.0f || (d == 0.0f && ((int)n & 1)) ? 1.0f : 0.0f);
  return __float_as_uint(__fadd_rn(copysignf(c, x), 12582912.0f));
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
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int c, int cols, bool vec) {
  Chunk<T> k;
  if (vec && c <= cols - 8) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(row + c)[i];
      k.w[4 * i] = u.x; k.w[4 * i + 1] = u.y; k.w[4 * i + 2] = u.z; k.w[4 * i + 3] = u.w;
    }
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) k.w[i] = c < cols - i ? reinterpret_cast<const uint32_t*>(row)[c + i] : 0u;
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      k.w[i] = (c < cols - 2 * i ? (uint32_t)h[c + 2 * i] : 0u) | (c < cols - 2 * i - 1 ? (uint32_t)h[c + 2 * i + 1] << 16 : 0u);
  }
  return k;
}

// The larger of `top` and |x|; NaN if one is (bf16: two numbers in a word).
__device__ __forceinline__ uint32_t max_abs(uint32_t top, uint32_t x) {
  asm("{\n\t.reg .f32 a;\n\tabs.f32 a, %1;\n\tmax.NaN.f32 %0, %2, a;\n\t}" : "=r"(top) : "r"(x), "r"(top));
  return top;
}
__device__ __forceinline__ uint32_t max_abs2(uint32_t top, uint32_t x) {
  asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %1;\n\tmax.NaN.bf16x2 %0, %2, a;\n\t}" : "=r"(top) : "r"(x), "r"(top));
  return top;
}

// Largest |x| as fp32 bits (they order like the values); NaN and infinities give kInf or more.
template <typename T>
__device__ __forceinline__ uint32_t chunk_top(const Chunk<T>& k, uint32_t top) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max_abs(top, k.w[i]);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_abs2(m, k.w[i]);
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
// Four at a time where something is open: code_at_border, or code_exact for a line with s.a < 0.
__device__ __noinline__ uint32_t four_open(float x0, float x1, float x2, float x3, float a, float inv, float lo) {
  const LineScale s{a, inv, lo};
  if (a < 0.0f)
    return pack4((uint32_t)code_exact(x0, -a, inv), (uint32_t)code_exact(x1, -a, inv), (uint32_t)code_exact(x2, -a, inv),
                 (uint32_t)code_exact(x3, -a, inv));
  return pack4(code_at_border(x0, s), code_at_border(x1, s), code_at_border(x2, s), code_at_border(x3, s));
}
template <typename T>
__device__ __forceinline__ uint32_t four_codes(float x0, float x1, float x2, float x3, const LineScale& s) {
  uint32_t b0, b1, b2, b3;
  float border = 0.0f;
  code_bits<T>(x0, x1, s, b0, b1, border);
  code_bits<T>(x2, x3, s, b2, b3, border);
  if (s.a < 0.0f || border > 0.49996f) return four_open(x0, x1, x2, x3, s.a, s.inv, s.lo);
  return pack4(b0, b1, b2, b3);
}
template <typename T>
__device__ __forceinline__ uint2 chunk_codes(const Chunk<T>& k, const LineScale& s) {
  return make_uint2(four_codes<T>(k.get(0), k.get(1), k.get(2), k.get(3), s),
                    four_codes<T>(k.get(4), k.get(5), k.get(6), k.get(7), s));
}

// Eight codes; the bytes of columns >= cols are not written.
__device__ __forceinline__ void store_codes(int8_t* row, int c, int cols, uint2 w) {
  if (c <= cols - 8) {
    *reinterpret_cast<uint2*>(row + c) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c < cols - i) row[c + i] = (int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}

// ---------------------------------------------------------------- rows
// GROUP threads take a row at a time and hold it, four chunks each at most, between the maximum
// and the codes, so it is read once; the next row is loaded before the work on one begins
// (without that a block waited for its loads most of the time, 2 us more at 8192 x 4096 bf16).
// A block is one group, or eight where a group is a warp, and goes on to further rows.  8192 x 4096 bf16
// takes 17 us, 5.9 TB/s of elements and codes; 4096 x 14336 fp32 47.4, 6.2.
//   TOPS: a thread meets the same columns in every row; it keeps their maxima in shared memory
// (its own words, 64 registers a thread are full), and the block joins them into one of kCopies
// copies of `tops` by integer atomicMax, whose order does not matter.  Many copies and few blocks,
// since blocks that meet at an address wait for one another (888 blocks and one copy took 10 us
// longer than the rows alone).  codes == nullptr: only that.
constexpr int kCopies = METIS_INT8_SCRATCH_COPIES;

// Larger of the magnitudes in `top` and in a word of a chunk (bf16 two to a word; their bits order
// like the values).
template <typename T>
__device__ __forceinline__ uint32_t word_top(uint32_t top, uint32_t w) {
  if constexpr (sizeof(T) == 2) return max_abs2(top, w);
  else return max_abs(top, w);
}
template <int GROUP>
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(GROUP) : "memory");
}

// A chunk with entries that are not finite: they are left out and their columns marked.
template <typename T>
__device__ __noinline__ Chunk<T> mark_nonfinite(Chunk<T> k, int c, uint32_t* marks, uint32_t* status) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if ((__float_as_uint(k.get(j)) & 0x7FFFFFFFu) >= kInf) {
      marks[c + j] = 1;
      if constexpr (sizeof(T) == 4) k.w[j] = 0;
      else k.w[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
    }
  raise_status(status, METIS_DEV_NONFINITE);
  return k;
}

// Threads of a block (several groups) and blocks of an SM: what the registers allow.
template <int GROUP, bool TOPS>
constexpr int kRowBlock = TOPS ? (GROUP == 512 ? 512 : 256) : GROUP == 32 ? kThreads : GROUP;
template <typename T, int GROUP, int HELD, bool TOPS>
constexpr int kRowBlocks = (HELD * (int)sizeof(T) == 16 ? 640 : TOPS ? 768 : 1024) / kRowBlock<GROUP, TOPS>;

template <typename T, int GROUP, int HELD, bool TOPS>
__global__ void __launch_bounds__(kRowBlock<GROUP, TOPS>, kRowBlocks<T, GROUP, HELD, TOPS>)
    quantize_i8_rows_kernel(const T* __restrict__ M, int64_t rows, int cols, int64_t ld, int8_t* __restrict__ codes,
                            int64_t ldq, float* __restrict__ scales, uint32_t* __restrict__ tops, int64_t tops_pitch,
                            uint32_t* __restrict__ marks, uint32_t* status) {
  constexpr int BLOCK = kRowBlock<GROUP, TOPS>, GROUPS = BLOCK / GROUP, VECS = (int)sizeof(T) / 2;
  __shared__ uint32_t part[2][2][BLOCK / 32];
  extern __shared__ __align__(16) uint4 col[];   // [HELD][VECS][BLOCK]
  tc::grid_dependency_wait();     // only now, so that whatever follows early finds all before this complete
  tc::grid_launch_dependents();
  const int t = threadIdx.x % GROUP, group = threadIdx.x / GROUP;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  int64_t r = (int64_t)blockIdx.x * GROUPS + group;

  auto load_row = [&](int64_t r, Chunk<T> (&k)[HELD]) {
    const T* row = M + r * ld;
    const bool vec = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
#pragma unroll
    for (int i = 0; i < HELD; ++i) k[i] = load_chunk(row, (i * GROUP + t) * 8, cols, vec);
  };
  auto over_row = [&](uint32_t top, uint32_t* slot) {
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (GROUP > 32) {
      if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = top;
      if constexpr (GROUPS == 1) __syncthreads();
      else group_sync<GROUP>(group);
#pragma unroll
      for (int i = 0; i < GROUP / 32; ++i) top = max(top, slot[group * (GROUP / 32) + i]);
    }
    return top;
  };
  auto add_to_columns = [&](int i, const Chunk<T>& k) {
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      uint4& at = col[(i * VECS + v) * BLOCK + threadIdx.x];
      uint4 m = at;
      m.x = word_top<T>(m.x, k.w[4 * v]);
      m.y = word_top<T>(m.y, k.w[4 * v + 1]);
      m.z = word_top<T>(m.z, k.w[4 * v + 2]);
      m.w = word_top<T>(m.w, k.w[4 * v + 3]);
      at = m;
    }
  };

  if constexpr (TOPS)
    for (int i = 0; i < HELD * VECS; ++i) col[i * BLOCK + threadIdx.x] = make_uint4(0, 0, 0, 0);
  Chunk<T> next[HELD];
  if (r < rows) load_row(r, next);
  for (int turn = 0; r < rows; r += step, turn ^= 1) {
    Chunk<T> held[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = next[i];
    if (r + step < rows) load_row(r + step, next);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < HELD; ++i) top = chunk_top(held[i], top);
    if constexpr (TOPS) {
      if (top < kInf) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) add_to_columns(i, held[i]);
      } else {
#pragma unroll
        for (int i = 0; i < HELD; ++i) add_to_columns(i, mark_nonfinite(held[i], (i * GROUP + t) * 8, marks, status));
      }
      if (!codes) continue;
    }
    top = over_row(top, part[turn][0]);
    const bool bad = top >= kInf;      // the same in the whole group
    if (bad) {
      top = 0;
#pragma unroll
      for (int i = 0; i < HELD; ++i) top = chunk_finite_top(held[i], top);
      top = over_row(top, part[turn][1]);
    }
    const LineScale s = line_scale(top, bad);
    if (t == 0) {
      scales[r] = scale_of(s);
      if (bad) raise_status(status, METIS_DEV_NONFINITE);
    }
    int8_t* out = codes + r * ldq;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int c = (i * GROUP + t) * 8;
      if (c < cols) store_codes(out, c, cols, chunk_codes(held[i], s));
    }
  }
  if constexpr (TOPS) {
    __syncthreads();
    uint32_t* const copy = tops + (int64_t)(blockIdx.x % kCopies) * tops_pitch;
    constexpr int PER_WORD = 4 / (int)sizeof(T);
    for (int c = threadIdx.x; c < cols; c += BLOCK) {
      const int chunk = c >> 3, i = chunk / GROUP, word = (c & 7) / PER_WORD;   // word of the chunk
      const uint32_t* at = reinterpret_cast<const uint32_t*>(col + (i * VECS + word / 4) * BLOCK + chunk % GROUP) + (word & 3);
      uint32_t m = 0;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) m = word_top<T>(m, at[g * GROUP * 4]);
      if constexpr (sizeof(T) == 2) m = (c & 1) ? m & 0xFFFF0000u : m << 16;
      if (m) atomicMax(&copy[c], m);
    }
  }
}

// A row longer than a group holds: read twice, the second time from L2 if it fits there.
template <typename T>
__global__ void __launch_bounds__(512) quantize_i8_long_rows_kernel(const T* __restrict__ M, int cols, int64_t ld,
                                                                    int8_t* __restrict__ codes, int64_t ldq,
                                                                    float* __restrict__ scales, uint32_t* status) {
  __shared__ uint32_t part[2][16];
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  const int64_t r = blockIdx.x;
  const T* row = M + r * ld;
  const bool vec = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
  auto over_row = [&](bool finite_only) {
    uint32_t top = 0;
    for (uint32_t c = threadIdx.x * 8; c < (uint32_t)cols; c += 512 * 8) {
      const Chunk<T> k = load_chunk(row, c, cols, vec);
      top = finite_only ? chunk_finite_top(k, top) : chunk_top(k, top);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) part[finite_only][threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, part[finite_only][i]);
    return top;
  };
  uint32_t top = over_row(false);
  const bool bad = top >= kInf;
  if (bad) top = over_row(true);
  const LineScale s = line_scale(top, bad);
  if (threadIdx.x == 0) {
    scales[r] = scale_of(s);
    if (bad) raise_status(status, METIS_DEV_NONFINITE);
  }
  for (uint32_t c = threadIdx.x * 8; c < (uint32_t)cols; c += 512 * 8)
    store_codes(codes + r * ldq, c, cols, chunk_codes(load_chunk(row, c, cols, vec), s));
}

// ---------------------------------------------------------------- columns
// The codes of the columns from their maxima: a tile of 128 bytes of ROWS rows goes to shared
// memory, all of it on its way at once (cp.async), also under the tail of the kernel that makes
// the maxima.  Then a thread takes a word of a row (two columns bf16, one fp32) in 16
// consecutive rows, so its codes are 16 bytes of a column each; the lanes of a warp are 4 words
// by 8 such pieces, so a column leaves as 128 bytes.  16 bytes of padding after 16 rows keep
// the pieces on different banks.  Tiles go from the last row to the first: the last rows read
// before are what L2 still holds.  With the rows' pass 8192 x 4096 bf16 takes 38.5 us, 4096 x 14336 fp32 108
// (34 and 88 where only columns are asked for): two readings, and 60% of the issue slots.
//   (One reading instead of two, by clusters that keep strips of columns in shared memory while
// their maxima are joined, took 36 us or more at 8192 x 4096 bf16 in all forms tried: a block
// waited most of its time for the join.)
constexpr int kPiece = 16, kRowBytes = 128;
constexpr int kPieceBytes = kPiece * kRowBytes + 16;

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <typename T, int ROWS>
__global__ void __launch_bounds__(kThreads, 4) quantize_i8_cols_kernel(const T* __restrict__ M, int64_t rows, int64_t cols,
                                                                       int64_t ld, int8_t* __restrict__ codes, int64_t ldq,
                                                                       float* __restrict__ scales, const uint32_t* tops,
                                                                       const uint32_t* marks) {
  constexpr int COLS = kRowBytes / (int)sizeof(T), PER_WORD = 4 / (int)sizeof(T);
  __shared__ __align__(16) uint8_t data[ROWS / kPiece * kPieceBytes];
  const int64_t strips = (cols + COLS - 1) / COLS, c0 = (blockIdx.x % strips) * COLS;
  const int64_t tile = (rows + ROWS - 1) / ROWS - 1 - blockIdx.x / strips, r0 = tile * ROWS;
  const int n = (int)min((int64_t)ROWS, rows - r0);
  const bool aligned = ((reinterpret_cast<uintptr_t>(M) | (uintptr_t)(ld * (int64_t)sizeof(T))) & 15u) == 0;
  if (aligned && c0 + COLS <= cols) {
    const int chunk = threadIdx.x & 7;
    const T* src = M + (r0 + (threadIdx.x >> 3)) * ld + c0 + chunk * (16 / (int)sizeof(T));
    for (int r = threadIdx.x >> 3; r < n; r += kThreads / 8, src += (kThreads / 8) * ld)
      copy_async16(data + (r / kPiece) * kPieceBytes + (r % kPiece) * kRowBytes + chunk * 16, src);
  } else {
    const int j = threadIdx.x % COLS;
    const T* src = M + (r0 + threadIdx.x / COLS) * ld + c0 + j;
    if (c0 + j < cols)
#pragma unroll 8
      for (int r = threadIdx.x / COLS; r < n; r += kThreads / COLS, src += (kThreads / COLS) * ld)
        // from L2, as cp.async.cg: read before the wait, when this SM's cache may hold an older matrix
        *(reinterpret_cast<T*>(data + (r / kPiece) * kPieceBytes + (r % kPiece) * kRowBytes) + j) = __ldcg(src);
  }
  tc::grid_dependency_wait();   // for the maxima
  tc::grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int word = warp * 4 + (lane & 3);
  const int64_t c = c0 + word * PER_WORD;
  LineScale ls[PER_WORD];
#pragma unroll
  for (int e = 0; e < PER_WORD; ++e) {
    uint32_t top = 0;
    if (c + e < cols)
#pragma unroll
      for (int i = 0; i < kCopies; ++i) top = max(top, tops[i * cols + c + e]);
    ls[e] = line_scale(top, c + e < cols && marks[c + e] != 0);
    if (tile == 0 && lane < 4 && c + e < cols) scales[c + e] = scale_of(ls[e]);
  }
  copy_async_wait_all();
  __syncthreads();
#pragma unroll 1
  for (int piece = lane >> 2; piece < ROWS / kPiece; piece += 8) {
    const int left = n - piece * kPiece;
    if (left <= 0) break;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(data + piece * kPieceBytes) + word;
    uint32_t out[PER_WORD][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = w[(4 * i + j) * (kRowBytes / 4)];
#pragma unroll
      for (int e = 0; e < PER_WORD; ++e) {
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(sizeof(T) == 4 ? x[j] : e ? x[j] & 0xFFFF0000u : x[j] << 16);
        out[e][i] = four_codes<T>(f[0], f[1], f[2], f[3], ls[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < PER_WORD; ++e) {
      if (c + e >= cols) continue;
      int8_t* dst = codes + (c + e) * ldq + r0 + piece * kPiece;
      if (left >= kPiece) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(out[e][0], out[e][1], out[e][2], out[e][3]);
      } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
          if (i < left) dst[i] = (int8_t)(out[e][i >> 2] >> (8 * (i & 3)));
      }
    }
  }
}

// Zeroes two stretches of words.  A kernel, not a memset: the next one is launched under it.
__global__ void __launch_bounds__(kThreads) clear_i8_scratch_kernel(uint32_t* a, int64_t na, uint32_t* b, int64_t nb) {
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < na + nb; i += (int64_t)gridDim.x * kThreads)
    *(i < na ? a + i : b + (i - na)) = 0;
}

// ---------------------------------------------------------------- launches
// All kernels here are launched so that they may start under the tail of the one before.
template <typename T, int GROUP, int HELD, bool TOPS>
cudaError_t launch_rows(const T* M, int64_t rows, int64_t cols, int64_t ld, const metis_int8* q, uint32_t* tops,
                        int64_t pitch, uint32_t* marks, uint32_t* status, int sm_count, cudaStream_t st) {
  constexpr int BLOCK = kRowBlock<GROUP, TOPS>, GROUPS = BLOCK / GROUP;
  constexpr int SMEM = TOPS ? HELD * (int)sizeof(T) / 2 * BLOCK * 16 : 0;
  const int64_t blocks = std::min<int64_t>((rows + GROUPS - 1) / GROUPS, (int64_t)sm_count * kRowBlocks<T, GROUP, HELD, TOPS>);
  auto kern = quantize_i8_rows_kernel<T, GROUP, HELD, TOPS>;
  if (SMEM > 48 * 1024 - 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
  }
  return launch_early(kern, blocks, BLOCK, SMEM, st, M, rows, (int)cols, ld, q ? q->codes : nullptr, q ? q->ld : 0,
                      q ? q->scales : nullptr, tops, pitch, marks, status);
}

// A thread holds 64 bytes of a row, or 128 for the longest fp32 rows: the smallest group that
// holds a row; where rows are too few to fill the SMs, the largest that has a chunk or two for
// each thread.
template <typename T, bool TOPS>
cudaError_t run_rows(const T* M, int64_t rows, int64_t cols, int64_t ld, const metis_int8* q, uint32_t* tops, int64_t pitch,
                     uint32_t* marks, uint32_t* status, int sm_count, cudaStream_t st) {
  constexpr int HELD = 8 / (int)sizeof(T);
  const int64_t chunks = (cols + 7) / 8;
  const int64_t need = rows < 4 * (int64_t)sm_count ? std::min<int64_t>(512, chunks / 2) : 0;
  const int64_t threads = std::max(need, (chunks + HELD - 1) / HELD);
#define METIS_ROWS(G, H) launch_rows<T, G, H, TOPS>(M, rows, cols, ld, q, tops, pitch, marks, status, sm_count, st)
  if (threads <= 32) return METIS_ROWS(32, HELD);
  if (threads <= 64) return METIS_ROWS(64, HELD);
  if (threads <= 128) return METIS_ROWS(128, HELD);
  if (threads <= 256) return METIS_ROWS(256, HELD);
  if (threads <= 512) return METIS_ROWS(512, HELD);
  return METIS_ROWS(512, 4);
#undef METIS_ROWS
}

constexpr int64_t kMostHeld = 512 * 4 * 8;   // columns

template <typename T>
cudaError_t run_quantize(const T* M, int64_t rows, int64_t cols, int64_t ld, const metis_int8* row, const metis_int8* col,
                         uint32_t* status, int sm_count, cudaStream_t st) {
  uint32_t *tops = nullptr, *marks = nullptr;
  cudaError_t e = cudaSuccess;
  if (col) {
    tops = col->scratch;
    marks = col->scratch + kCopies * cols;
  }
  if (row && cols > kMostHeld) {
    e = launch_early(quantize_i8_long_rows_kernel<T>, rows, 512, 0, st, M, (int)cols, ld, row->codes, row->ld, row->scales, status);
    if (e != cudaSuccess) return e;
  }
  if (!col) return cols > kMostHeld ? e : run_rows<T, false>(M, rows, cols, ld, row, nullptr, 0, nullptr, status, sm_count, st);
  if (row && cols <= kMostHeld) {
    e = run_rows<T, true>(M, rows, cols, ld, row, tops, cols, marks, status, sm_count, st);
  } else {   // only the maxima: columns in spans
    for (int64_t c = 0; c < cols && e == cudaSuccess; c += kMostHeld)
      e = run_rows<T, true>(M + c, rows, std::min(kMostHeld, cols - c), ld, nullptr, tops + c, cols, marks + c, status, sm_count, st);
  }
  if (e != cudaSuccess) return e;
  constexpr int COLS = kRowBytes / (int)sizeof(T);
  const int64_t strips = (cols + COLS - 1) / COLS;
  auto launch = [&](auto kern, int64_t tile) {
    return launch_early(kern, strips * ((rows + tile - 1) / tile), kThreads, 0, st, M, rows, cols, ld, col->codes, col->ld,
                        col->scales, (const uint32_t*)tops, (const uint32_t*)marks);
  };
  // Rows of a tile: 256, or half that where there would be fewer than two blocks for an SM.  Both
  // orientations, 128 against 256: 1001 x 1333 bf16 10.3 us, 13.0; 2048 x 2048 10.0, 10.4; 4096 x 2048 14.3,
  // 13.8; 8192 x 4096 42.9, 38.5.
  if (strips * ((rows + 255) / 256) < 2 * (int64_t)sm_count) return launch(quantize_i8_cols_kernel<T, 128>, 128);
  return launch(quantize_i8_cols_kernel<T, 256>, 256);
}

}  // namespace

cudaError_t clear_int8_scratch(const metis_int8* a, const metis_int8* b, int sm_count, cudaStream_t st) {
  const int64_t na = a ? (int64_t)METIS_INT8_SCRATCH * a->outer : 0, nb = b ? (int64_t)METIS_INT8_SCRATCH * b->outer : 0;
  if (na + nb == 0) return cudaSuccess;
  const int64_t blocks = std::min<int64_t>((na + nb + kThreads - 1) / kThreads, 2 * (int64_t)sm_count);
  return launch_early(clear_i8_scratch_kernel, blocks, kThreads, 0, st, a ? a->scratch : nullptr, na, b ? b->scratch : nullptr, nb);
}

cudaError_t launch_quantize_i8(const void* M, bool bf16, int64_t rows, int64_t cols, int64_t ld, const metis_int8* row,
                               const metis_int8* col, uint32_t* status, int sm_count, cudaStream_t st) {
  if (bf16)
    return run_quantize(static_cast<const __nv_bfloat16*>(M), rows, cols, ld, row, col, status, sm_count, st);
  return run_quantize(static_cast<const float*>(M), rows, cols, ld, row, col, status, sm_count, st);
}

}  // namespace metis
