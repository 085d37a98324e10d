// AdamW (Loshchilov and Hutter, "Decoupled Weight Decay Regularization") over many tensors
// in one launch, with the moments in 32 bits or in 8.
//
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit moments: 128 consecutive elements of a tensor share an exponent byte
// E = 127 + floor(log2(max)) of the block (at least 16), and each element is a small float
// with 3 mantissa bits and gradual underflow below it:
//   m: sign, 4 exponent bits:  |m| = c u (c < 8) or (8 + c % 8) 2^(c / 8 - 1) u, u = 2^(E - 127 - 17)
//   v: 5 exponent bits, u = 2^(E - 127 - 33); a positive v is held at u at least, because a
//      v of zero beside a nonzero m would make a step of m / eps.
// v spans 33 octaves below the block's largest, so 16 in its root.  The shared exponent is a
// power of two, so decoding is exact and encoding rounds once, from the fp64 value of the
// formula.  That value is defined with every product and sum rounded (none fused): coarse
// operands meet borders between codes exactly -- (9 m + g) / 10 of a 4-bit m and a bf16 g does
// in one case of some hundred -- and a fused sum would decide those the other way.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "device_common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace metis {
namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 1024;           // elements a block takes at once: a state block for each warp
constexpr int kStateBlock = 128;      // elements that share an exponent
constexpr int kMOctaves = 15, kVOctaves = 31;

struct Tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* me;
  uint8_t* ve;
  int64_t n;
};

struct Coef {
  double b1, b2, lr, wd, eps;
  int64_t step;
  const float* lr_dev;        // nullable: the learning rate is read on the device
  const int64_t* step_dev;    // nullable: t is read on the device
  uint64_t seed;
};

template <int CAP>
struct Table {
  Coef c;
  int count;
  int64_t chunks;             // of all tensors
  int units;                  // of a chunk, which a block handles at a time
  uint32_t* status;
  uint2 keys[10];             // Philox round keys
  uint32_t id[CAP];           // random stream of each tensor
  int64_t first[CAP];         // first chunk of each tensor
  Tensor t[CAP];
};

// What a step needs of its coefficients, in fp32.
struct Step {
  float decay, size, rbc2, eps;
  float b1, b1_low;       // beta1: its upper 20 bits and the rest
  float a1, a1_low;       // 1 - beta1: nearest and the rest
  float b2, a2;           // beta2 and 1 - beta2
  bool tiny;              // eps does not hide the root of a subnormal v
  uint32_t t;
};

// 1 - b^t by repeated squaring in fp64.
__host__ __device__ inline double one_minus_power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return 1.0 - r;
}

__device__ Step make_step(const Coef& c) {
  const int64_t t = c.step_dev ? *c.step_dev : c.step;
  const double lr = c.lr_dev ? (double)*c.lr_dev : c.lr;
  Step s;
  s.decay = (float)(1.0 - lr * c.wd);
  s.size = (float)(lr / one_minus_power(c.b1, t));
  s.rbc2 = (float)(1.0 / sqrt(one_minus_power(c.b2, t)));
  s.eps = (float)c.eps;
  if (s.eps == 0.0f && c.eps > 0.0) s.eps = __uint_as_float(1u);   // the smallest fp32: m = v = 0 stays 0 / eps
  s.b1 = __uint_as_float(__float_as_uint((float)c.b1) & ~15u);
  s.b1_low = (float)(c.b1 - (double)s.b1);
  s.a1 = (float)(1.0 - c.b1);
  s.a1_low = (float)((1.0 - c.b1) - (double)s.a1);
  s.tiny = !(c.eps >= 1e-11);
  s.b2 = (float)c.b2;
  s.a2 = (float)(1.0 - c.b2);
  s.t = (uint32_t)t;
  return s;
}

// Root and reciprocal within 2^-23 and 2^-22.  Flushing a subnormal v (root below 2^-63) to 0 does
// not show beside an eps of 1e-11; with a smaller one (TINY) the slower forms keep it.
template <bool TINY>
__device__ __forceinline__ float stepped(float p, float m, float v, const Step& s) {
  float root, q;
  if constexpr (!TINY) {
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(fmaf(root, s.rbc2, s.eps)));
    q *= m;
  } else {
    asm("sqrt.approx.f32 %0, %1;" : "=f"(root) : "f"(v));
    q = __fdiv_rn(m, fmaf(root, s.rbc2, s.eps));
  }
  return fmaf(-s.size, q, p * s.decay);
}

// The words of one counter (philox10 with its round keys from the table, which saves their sums).
__device__ __forceinline__ Words4 stream_words(const uint2 (&keys)[10], uint32_t tag, uint32_t step, uint64_t q) {
  uint32_t c0 = (uint32_t)q, c1 = (uint32_t)(q >> 32), c2 = tag, c3 = step;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ keys[r].x;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ keys[r].y;
    c3 = (uint32_t)a;
  }
  return Words4{{c0, c1, c2, c3}};
}

// Four consecutive elements as they are in memory; unpacked where they are used, so that a load
// ahead is not waited for.
template <typename T>
struct __align__(4 * sizeof(T)) Four {
  uint32_t w[(int)sizeof(T)];
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    else return __uint_as_float((j & 1) ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
  }
};

// From element i on of a tensor of n; what is beyond reads as 0.
template <typename T>
__device__ __forceinline__ Four<T> load4(const T* a, int64_t i, int64_t n, bool vec) {
  Four<T> x;
  if (vec && i + 4 <= n) {
    if constexpr (sizeof(T) == 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(a + i);
      x.w[0] = u.x; x.w[1] = u.y; x.w[2] = u.z; x.w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(a + i);
      x.w[0] = u.x; x.w[1] = u.y;
    }
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x.w[j] = i + j < n ? __float_as_uint(a[i + j]) : 0u;
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(a);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      x.w[j] = (i + 2 * j < n ? (uint32_t)h[i + 2 * j] : 0u) | (i + 2 * j + 1 < n ? (uint32_t)h[i + 2 * j + 1] << 16 : 0u);
  }
  return x;
}

__device__ __forceinline__ void store4(float* a, int64_t i, int64_t n, bool vec, const float (&x)[4]) {
  if (vec && i + 4 <= n) {
    *reinterpret_cast<float4*>(a + i) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) a[i + j] = x[j];
  }
}

// bf16 parameters: nearest-even, or stochastic with the low 16 bits of the element's word
// (a step far below half a unit of the parameter would be lost by the nearest).
__device__ __forceinline__ void store4(__nv_bfloat16* a, int64_t i, int64_t n, bool vec, const float (&x)[4],
                                       bool stochastic, const Words4& w) {
  uint16_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t b = __float_as_uint(x[j]);
    if (stochastic && (b & 0x7F800000u) != 0x7F800000u)
      h[j] = (uint16_t)((b + (w.w[j] & 0xFFFFu)) >> 16);
    else
      h[j] = __bfloat16_as_ushort(__float2bfloat16_rn(x[j]));
  }
  if (vec && i + 4 <= n) {
    *reinterpret_cast<uint2*>(a + i) =
        make_uint2((uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) a[i + j] = __ushort_as_bfloat16(h[j]);
  }
}

__device__ __forceinline__ uint32_t load_codes(const uint8_t* a, int64_t i, int64_t n, bool vec) {
  if (vec && i + 4 <= n) return *reinterpret_cast<const uint32_t*>(a + i);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) w |= (uint32_t)a[i + j] << (8 * j);
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* a, int64_t i, int64_t n, bool vec, uint32_t w) {
  if (vec && i + 4 <= n) {
    *reinterpret_cast<uint32_t*>(a + i) = w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) a[i + j] = (uint8_t)(w >> (8 * j));
  }
}

__device__ __forceinline__ double power2(int e) { return __hiloint2double((e + 1023) << 20, 0); }   // -1022 .. 1023
__device__ __forceinline__ float power2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 .. 127

// ---- the moments in fp64, by their definition -------------------------------------
// A code's magnitude is the fp64 number with bits code << 49 (exponent field code / 8, so
// that gradual underflow is the format's own) times 2^(1022 + E - 127 - octaves + 1).
__device__ __forceinline__ double decode64(uint32_t code, int top, int octaves) {
  return __hiloint2double((int)(code << 17), 0) * power2(1000) * power2(22 + top - octaves + 1);
}
__device__ __forceinline__ double first_moment(uint32_t code, int top, float g, double b1) {
  const double old = decode64(code & 127u, top, kMOctaves);
  return __dadd_rn(__dmul_rn(b1, code > 127u ? -old : old), __dmul_rn(1.0 - b1, (double)g));
}
__device__ __forceinline__ double second_moment(uint32_t code, int top, float g, double b2) {
  return __dadd_rn(__dmul_rn(b2, decode64(code, top, kVOctaves)), __dmul_rn(1.0 - b2, __dmul_rn((double)g, (double)g)));
}
__device__ __forceinline__ int exponent_field(double x) { return (__double2hiint(x) >> 20) & 0x7FF; }

// The code of a finite x >= 0 from t = x / u.  From 8 on, 3 mantissa bits are kept by an integer
// addition to the fp64 number (its exponent and upper mantissa bits count the codes); below
// 8 the grid's step is 1.
template <bool SR>
__device__ __forceinline__ uint32_t encode64(double x, int top, int octaves, uint32_t field) {
  const double t = x * power2(octaves + 2 - top);
  if (t < 8.0)
    return (uint32_t)(SR ? __double2int_rd(t + ((double)field + 0.5) * (1.0 / 65536.0)) : __double2int_rn(t));
  const unsigned long long b = (unsigned long long)__double_as_longlong(t);
  unsigned long long r;
  if (SR)
    r = ((unsigned long long)field << 33) + (1ull << 32);                 // (field + 1/2) 2^-16 of a step
  else
    r = ((1ull << 48) - 1) + ((b >> 49) & 1);                             // nearest, ties to even
  return min((uint32_t)((b + r) >> 49) - (1026u * 8u - 8u), 8u * octaves + 7u);   // 8.0 has the exponent field 1026
}

// The same with the block's old and new exponents, for one element.
template <bool SR>
__device__ __noinline__ uint32_t exact_codes(uint32_t cm, uint32_t cv, int old_tm, int old_tv, int tm, int tv, float g,
                                             double b1, double b2, uint32_t word) {
  const double m = first_moment(cm, old_tm, g, b1), v = second_moment(cv, old_tv, g, b2);
  // an element whose gradient was not finite (its parameter is NaN now) restarts from zero
  if (exponent_field(m) == 0x7FF || exponent_field(v) == 0x7FF) return 0u;
  uint32_t c = encode64<SR>(fabs(m), tm, kMOctaves, word & 0xFFFFu);
  if (c && m < 0.0) c |= 128u;
  return c | max(encode64<SR>(v, tv, kVOctaves, word >> 16), v > 0.0 ? 1u : 0u) << 8;
}
__device__ __noinline__ float2 exact_moments(uint32_t cm, uint32_t cv, int old_tm, int old_tv, float g, double b1, double b2) {
  return make_float2((float)first_moment(cm, old_tm, g, b1), (float)second_moment(cv, old_tv, g, b2));
}
__device__ __noinline__ uint32_t exact_fields(uint32_t cm, uint32_t cv, int old_tm, int old_tv, float g, double b1, double b2) {
  const int em = exponent_field(first_moment(cm, old_tm, g, b1)), ev = exponent_field(second_moment(cv, old_tv, g, b2));
  return (em == 0x7FF ? 0u : (uint32_t)em) | (ev == 0x7FF ? 0u : (uint32_t)ev) << 16;
}
// Exponent byte - 127 of a block from the largest fp64 exponent field of its elements.
__device__ __forceinline__ int block_top(int field) { return min(max(field - 1023, -111), 127); }

// ---- the same in fp32 with a bound on the error -----------------------------------
// In fp64 throughout a step of 71 M elements took 611 us.  Instead the moments are taken in fp32,
// the first from two-word coefficients and an exact sum, so that both lie within three units of
// their last place of the fp64 values; where a border between codes is that near (one element
// in 10^5 of an fp32 gradient; a bf16 one meets borders exactly, one in 300) the fp64 route
// decides.
//   That takes a new exponent of the block at most kDrop octaves below the old.  The first moment's error
// besides its two roundings (one unit together) is below 2^-43 |b1 m|, from the rest of beta1 and the sum
// of the remainders, so below 2^(t_old - 42) in a block of exponent t_old; the unit of its smallest codes
// is 2^(t_new - 37).  Six octaves make that two units; where terms cancel further the fp64 route decides.
//   A magnitude is scaled so that the lowest normal octave of the codes is fp32's own: its bits
// count the codes in steps of 2^20, gradual underflow included, and what is added to round up is
// (field + 1/2) 2^-16 of a step, or to nearest half a step, less a unit unless the code is odd.
template <bool SR>
__device__ __forceinline__ uint32_t rounded(uint32_t bits, uint32_t field4) {   // field4 = 16 field
  return SR ? bits + field4 + 8u : bits + 0x7FFFFu + ((bits >> 20) & 1u);
}
constexpr uint32_t kNear = 4;   // units
constexpr int kDrop = 6;        // octaves

// One state block of 128 elements in a warp, four to a lane.
struct Block4 {
  float p[4], g[4];
  uint32_t cm, cv;
  int tm, tv;      // exponent bytes - 127
};

// The low eight bits above bit 20 of each, packed.
__device__ __forceinline__ uint32_t codes4(const uint32_t (&r)[4]) {
  const uint32_t a = __byte_perm(r[0], r[1], 0x7632) >> 4, b = __byte_perm(r[2], r[3], 0x7632) >> 4;
  return __byte_perm(a, b, 0x6420);
}

// Steps the block's parameters in place and gives its new codes and exponents.  Returns whether a
// gradient of the lane is not finite.
template <bool SR>
__device__ __forceinline__ bool step_block(Block4& x, const Step& s, double b1, double b2, const Words4& w) {
  // The fp32 route holds for exponents within these, where no scale leaves fp32's range and a
  // block's sums stay normal.
  const bool usual = x.tm <= 14 && x.tv <= 30;
  // the coefficients of the codes as they are: exact, the decoding factors are powers of two
  const float dm = power2f(min(x.tm, 14) + 112), dv = power2f(min(x.tv, 30) + 96);
  const Pair b1m(s.b1 * dm), b1m_low(-s.b1_low * dm), b2v(s.b2 * dv);
  float ym[4], yv[4];
  float hm = 0.0f;
  uint32_t hv = 0;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    // code j in the top byte, then its sign and magnitude in place
    auto old_m = [&](int j) { return __uint_as_float((uint32_t)((int)__byte_perm(x.cm, 0u, (j << 12) | 0x0444u) >> 4) & 0x87F00000u); };
    auto old_v = [&](int j) { return __uint_as_float(__byte_perm(x.cv, 0u, (j << 12) | 0x0444u) >> 4); };
    const Pair om(old_m(j), old_m(j + 1)), ov(old_v(j), old_v(j + 1)), g(x.g[j], x.g[j + 1]);
    // b1 m + (1 - b1) g: the first product exact within the sum (m has four bits, the coefficient
    // twenty), the second with its remainder (here negated); two roundings of the sum, so two units
    const Pair add = Pair(s.a1) * g;
    const Pair rest = fma2(b1m_low, om, fma2(Pair(-s.a1_low), g, fma2(Pair(-s.a1), g, add)));
    fma2(rest, Pair(-1.0f), fma2(b1m, om, add)).get(ym[j], ym[j + 1]);
    // five roundings: three units; (1 - b2) g first, since g g leaves fp32 from 1.8e19 on
    fma2(b2v, ov, Pair(s.a2) * g * g).get(yv[j], yv[j + 1]);
  }
  if (!usual) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = exact_moments((x.cm >> (8 * j)) & 255u, (x.cv >> (8 * j)) & 255u, x.tm, x.tv, x.g[j], b1, b2);
      ym[j] = y.x;
      yv[j] = y.y;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    hm = fmaxf(hm, fabsf(ym[j]));
    hv = max(hv, __float_as_uint(yv[j]));   // a NaN's bits lie above all others
  }
  if (!s.tiny) {
#pragma unroll
    for (int j = 0; j < 4; j += 2) {   // as stepped<false>
      float r0, r1, q0, q1;
      asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(yv[j]));
      asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(yv[j + 1]));
      fma2(Pair(r0, r1), Pair(s.rbc2), Pair(s.eps)).get(r0, r1);
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q0) : "f"(r0));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q1) : "f"(r1));
      const Pair q = Pair(q0, q1) * Pair(ym[j], ym[j + 1]);
      fma2(Pair(-s.size), q, Pair(x.p[j], x.p[j + 1]) * Pair(s.decay)).get(x.p[j], x.p[j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x.p[j] = stepped<true>(x.p[j], ym[j], yv[j], s);
  }
  // the block's exponents (bits of positive floats order like them), open next to a power of two, where
  // the first moments cancelled and beyond the range, where gradients that are not finite end up too
  const uint32_t top_m = __reduce_max_sync(0xffffffffu, __float_as_uint(hm)), top_v = __reduce_max_sync(0xffffffffu, hv);
  int tm = (int)(top_m >> 23) - 127, tv = (int)(top_v >> 23) - 127;
  const uint32_t edge = min((top_m + kNear) & 0x7FFFFFu, (top_v + kNear) & 0x7FFFFFu);
  const bool open = !usual || tm > 14 || tm < max(-60, x.tm - kDrop) || tv > 30 || tv < -60 || edge <= 2 * kNear;
  bool odd = false;
  uint32_t om, ov, redo = 0;
  if (open) {
    om = ov = 0;
    const bool some = (x.cm | x.cv) != 0u || x.g[0] != 0.0f || x.g[1] != 0.0f || x.g[2] != 0.0f || x.g[3] != 0.0f;
    odd = !isfinite(x.g[0]) || !isfinite(x.g[1]) || !isfinite(x.g[2]) || !isfinite(x.g[3]);
    if (!__any_sync(0xffffffffu, some)) {   // nothing there, and nothing new
      tm = tv = -111;
    } else {
      uint32_t f = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t e = exact_fields((x.cm >> (8 * j)) & 255u, (x.cv >> (8 * j)) & 255u, x.tm, x.tv, x.g[j], b1, b2);
        f = max(f & 0xFFFFu, e & 0xFFFFu) | max(f >> 16, e >> 16) << 16;
      }
      tm = block_top((int)__reduce_max_sync(0xffffffffu, f & 0xFFFFu));
      tv = block_top((int)__reduce_max_sync(0xffffffffu, f >> 16));
      redo = 0xFu;
    }
  } else {
    const float sm = power2f(-112 - tm), sv = power2f(-96 - tv);
    uint32_t rm[4], rv[4], near = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      rm[j] = rounded<SR>(__float_as_uint(fabsf(ym[j]) * sm), (w.w[j] << 4) & 0xFFFF0u);
      rv[j] = rounded<SR>(__float_as_uint(yv[j] * sv), (w.w[j] >> 12) & 0xFFFF0u);
      near = min(near, min(rm[j] * 4096u + kNear * 4096u, rv[j] * 4096u + kNear * 4096u));   // the low 20 bits
    }
    om = codes4(rm);
    om -= (om & 0x80808080u) >> 7;                   // 128, past the top code, becomes 127
    const uint32_t signs = __byte_perm(__byte_perm(__float_as_uint(ym[0]), __float_as_uint(ym[1]), 0x0073),
                                       __byte_perm(__float_as_uint(ym[2]), __float_as_uint(ym[3]), 0x0073), 0x5410);
    om |= (om + 0x7F7F7F7Fu) & signs & 0x80808080u;  // of codes that are not zero
    ov = codes4(rv);
    if (near <= 2 * kNear * 4096u) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (min(rm[j] * 4096u + kNear * 4096u, rv[j] * 4096u + kNear * 4096u) <= 2 * kNear * 4096u) redo |= 1u << j;
    }
    if ((ov - 0x01010101u) & ~ov & 0x80808080u) {    // a zero code of v: 1 where v is positive, 255 where it was 256
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!((ov >> (8 * j)) & 255u)) {
          if (rv[j] >> 28) ov |= 255u << (8 * j);
          else if (yv[j] > 0.0f) ov |= 1u << (8 * j);
          else if (x.g[j] != 0.0f || (x.cv >> (8 * j)) & 255u) redo |= 1u << j;   // fp64 may see more
        }
    }
  }
  while (redo) {
    const int j = __ffs(redo) - 1;
    redo &= redo - 1;
    const uint32_t word = j == 0 ? w.w[0] : j == 1 ? w.w[1] : j == 2 ? w.w[2] : w.w[3];
    const float gj = j == 0 ? x.g[0] : j == 1 ? x.g[1] : j == 2 ? x.g[2] : x.g[3];
    const uint32_t c = exact_codes<SR>((x.cm >> (8 * j)) & 255u, (x.cv >> (8 * j)) & 255u, x.tm, x.tv, tm, tv, gj, b1, b2, word);
    om = (om & ~(255u << (8 * j))) | (c & 255u) << (8 * j);
    ov = (ov & ~(255u << (8 * j))) | (c >> 8) << (8 * j);
  }
  x.cm = om;
  x.cv = ov;
  x.tm = tm;
  x.tv = tv;
  return odd;
}

// A tensor's arrays as the kernel walks them.  FAST: all are aligned and the chunk lies inside.
template <typename T, bool FAST>
struct View {
  T* p;
  const T* g;
  void* m;
  void* v;
  int64_t n;
  bool vec_p, vec_g, vec_s;
  __device__ __forceinline__ bool in(int64_t i) const { return FAST || i < n; }
  __device__ __forceinline__ Four<T> load_p(int64_t i) const { return load4(p, i, FAST ? i + 4 : n, FAST || vec_p); }
  __device__ __forceinline__ Four<T> load_g(int64_t i) const { return load4(g, i, FAST ? i + 4 : n, FAST || vec_g); }
  __device__ __forceinline__ void store(int64_t i, const float (&xp)[4], bool sr, const Words4& w) const {
    if constexpr (sizeof(T) == 4) store4(p, i, FAST ? i + 4 : n, FAST || vec_p, xp);
    else store4(p, i, FAST ? i + 4 : n, FAST || vec_p, xp, sr, w);
  }
};

// What a block has on its way in shared memory: each thread copies its own elements of the next two state
// blocks here and reads them back, so nothing but the copies is waited for.  Only fp32 to nearest, which
// waited for memory with one state block ahead in registers (71 M elements 246 us, 221 with the ring;
// four or six stages 1% and 4% more).  The others do not gain: fp32 stochastic 261 us, 263 with it;
// bf16 323, 341 stochastic, 301, 313 to nearest.
template <typename T>
struct Ring {
  static constexpr int STAGES = 3;
  Four<T> p[STAGES][kThreads], g[STAGES][kThreads];
  uint32_t cm[STAGES][kThreads], cv[STAGES][kThreads];
};
template <typename T, int BITS, bool SR>
constexpr bool kRing = BITS == 8 && sizeof(T) == 4 && !SR;
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_addr(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory"); }

// One chunk (elements base .. base + units * kUnit of a tensor).  Returns whether a gradient of the
// thread is not finite.
template <typename T, int BITS, bool SR, bool FAST, int CAP>
__device__ __forceinline__ bool run_chunk(const Table<CAP>& tab, int which, int64_t base, const View<T, FAST>& a, const Step& s,
                                          Ring<T>* ring) {
  bool bad = false;
  const uint32_t tag = stream_tag(tab.id[which], kPurposeState, 0);
  if constexpr (BITS == 32) {
    float* m = static_cast<float*>(a.m);
    float* v = static_cast<float*>(a.v);
    int64_t i = base + (int64_t)threadIdx.x * 4;
#pragma unroll 2
    for (int u = 0; u < tab.units; ++u, i += kUnit) {
      if (!a.in(i)) break;
      const Four<T> fp = a.load_p(i), fg = a.load_g(i);
      const Four<float> fm = load4(m, i, FAST ? i + 4 : a.n, FAST || a.vec_s), fv = load4(v, i, FAST ? i + 4 : a.n, FAST || a.vec_s);
      float xp[4], xm[4], xv[4], z = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float g = fg.get(j), old = fm.get(j);
        z = fmaf(g, 0.0f, z);
        xm[j] = fmaf(s.b1, old, fmaf(s.b1_low, old, s.a1 * g));
        xv[j] = fmaf(s.b2, fv.get(j), s.a2 * g * g);   // in this order: g g alone leaves fp32 from 1.8e19 on
        xp[j] = s.tiny ? stepped<true>(fp.get(j), xm[j], xv[j], s) : stepped<false>(fp.get(j), xm[j], xv[j], s);
      }
      bad |= z != z;
      store4(m, i, FAST ? i + 4 : a.n, FAST || a.vec_s, xm);
      store4(v, i, FAST ? i + 4 : a.n, FAST || a.vec_s, xv);
      Words4 w{};
      if (SR && sizeof(T) == 2) w = stream_words(tab.keys, tag | 1u, s.t, (uint64_t)i >> 2);
      a.store(i, xp, SR, w);
    }
  } else {
    constexpr bool AHEAD = FAST && kRing<T, BITS, SR>;
    uint8_t* m = static_cast<uint8_t*>(a.m);
    uint8_t* v = static_cast<uint8_t*>(a.v);
    uint8_t* me = tab.t[which].me;
    uint8_t* ve = tab.t[which].ve;
    // A warp takes `units` consecutive state blocks; their exponents are read and written at once, a
    // lane each.  (One at a time, stored beside others still to be read, they cost more than
    // all the rest: 71 M elements 466 us, 220 without them.)
    const int lane = threadIdx.x & 31;
    const int64_t first = base + (int64_t)(threadIdx.x >> 5) * tab.units * kStateBlock;
    if (!a.in(first)) return false;
    const int blocks = FAST ? tab.units : (int)min((int64_t)tab.units, (a.n - first + kStateBlock - 1) / kStateBlock);
    int64_t i = first + lane * 4;
    auto fetch = [&](int u, int64_t e) {   // elements e on, of the warp's state block u
      if (u < blocks) {
        const int at = u % Ring<T>::STAGES;
        copy_async<sizeof(Four<T>)>(&ring->p[at][threadIdx.x], a.p + e);
        copy_async<sizeof(Four<T>)>(&ring->g[at][threadIdx.x], a.g + e);
        copy_async<4>(&ring->cm[at][threadIdx.x], m + e);
        copy_async<4>(&ring->cv[at][threadIdx.x], v + e);
      }
      copy_async_commit();
    };
    if constexpr (AHEAD)
#pragma unroll
      for (int u = 0; u < Ring<T>::STAGES - 1; ++u) fetch(u, i + u * kStateBlock);
    const int64_t blk = first / kStateBlock + lane;
    const int old_me = lane < blocks ? (int)me[blk] - 127 : 0, old_ve = lane < blocks ? (int)ve[blk] - 127 : 0;
    int new_me = 0, new_ve = 0;
    struct {
      Four<T> p, g;
      uint32_t cm, cv;
    } next;
    auto load = [&](int64_t i) {
      next.p = a.load_p(i);
      next.g = a.load_g(i);
      next.cm = load_codes(m, i, FAST ? i + 4 : a.n, FAST || a.vec_s);
      next.cv = load_codes(v, i, FAST ? i + 4 : a.n, FAST || a.vec_s);
    };
    if constexpr (!AHEAD) load(i);
    for (int u = 0; u < blocks; ++u, i += kStateBlock) {
      if constexpr (AHEAD) {
        fetch(u + Ring<T>::STAGES - 1, i + (Ring<T>::STAGES - 1) * kStateBlock);
        copy_async_wait<Ring<T>::STAGES - 1>();
        const int at = u % Ring<T>::STAGES;
        next.p = ring->p[at][threadIdx.x];
        next.g = ring->g[at][threadIdx.x];
        next.cm = ring->cm[at][threadIdx.x];
        next.cv = ring->cv[at][threadIdx.x];
      }
      Block4 x;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x.p[j] = next.p.get(j);
        x.g[j] = next.g.get(j);
      }
      x.cm = next.cm;
      x.cv = next.cv;
      x.tm = __shfl_sync(0xffffffffu, old_me, u);
      x.tv = __shfl_sync(0xffffffffu, old_ve, u);
      if constexpr (!AHEAD)
        if (u + 1 < blocks) load(i + kStateBlock);
      Words4 w{};
      if (SR) w = stream_words(tab.keys, tag, s.t, (uint64_t)i >> 2);
      bad |= step_block<SR>(x, s, tab.c.b1, tab.c.b2, w);
      store_codes(m, i, FAST ? i + 4 : a.n, FAST || a.vec_s, x.cm);
      store_codes(v, i, FAST ? i + 4 : a.n, FAST || a.vec_s, x.cv);
      if (lane == u) {
        new_me = x.tm + 127;
        new_ve = x.tv + 127;
      }
      Words4 wp{};
      if (SR && sizeof(T) == 2) wp = stream_words(tab.keys, tag | 1u, s.t, (uint64_t)i >> 2);
      a.store(i, x.p, SR, wp);
    }
    if (lane < blocks) {
      me[blk] = (uint8_t)new_me;
      ve[blk] = (uint8_t)new_ve;
    }
  }
  return bad;
}

// 8-bit states: 71 M elements, all with gradients, take 221 us (fp32 to nearest), 261 (fp32 stochastic), 301 and 323
// (bf16).  Elements without gradients may settle on a border -- beta2 = 0.95 takes a v of code 10 to 9.5, and the
// nearest code is 10 again -- where the fp64 route decides in every step: with 2% of those 305 and 330 to nearest.
// Three blocks an SM leave 80 registers a thread, of which 4 to 12 bytes spill to nearest and 60 (bf16) or 76
// (fp32) with the words of the stochastic rounding; four blocks, or blocks of 128 threads at 5 to 7 an SM,
// were not faster.  Neither the issue slots (62%) nor the integer pipe (61%) nor HBM (39%) is full.
template <typename T, int BITS, bool SR, int CAP>
__global__ void __launch_bounds__(kThreads, BITS == 32 ? 5 : 3) adamw_kernel(const __grid_constant__ Table<CAP> tab) {
  __shared__ Step sh;
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  Ring<T>* const ring = reinterpret_cast<Ring<T>*>(ring_bytes);   // BITS == 8
  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  if (threadIdx.x == 0) sh = make_step(tab.c);
  __syncthreads();
  const Step s = sh;
  bool bad = false;
  for (int64_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    int lo = 0, hi = tab.count - 1;   // the last tensor whose first chunk is not beyond this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    const Tensor& t = tab.t[lo];
    const int64_t base = (chunk - tab.first[lo]) * tab.units * kUnit;
    const uintptr_t mask = sizeof(T) == 4 ? 15u : 7u, state_mask = BITS == 32 ? 15u : 3u;
    const bool vec_p = (reinterpret_cast<uintptr_t>(t.p) & mask) == 0, vec_g = (reinterpret_cast<uintptr_t>(t.g) & mask) == 0;
    const bool vec_s = ((reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) & state_mask) == 0;
    if (vec_p && vec_g && vec_s && base + (int64_t)tab.units * kUnit <= t.n)
      bad |= run_chunk<T, BITS, SR>(tab, lo, base, View<T, true>{static_cast<T*>(t.p), static_cast<const T*>(t.g), t.m, t.v, t.n, true, true, true}, s, ring);
    else
      bad |= run_chunk<T, BITS, SR>(tab, lo, base, View<T, false>{static_cast<T*>(t.p), static_cast<const T*>(t.g), t.m, t.v, t.n, vec_p, vec_g, vec_s}, s, ring);
  }
  if (bad) raise_status(tab.status, METIS_DEV_NONFINITE);
}

template <typename T, int BITS, bool SR, int CAP>
cudaError_t launch_cap(metis_ctx* ctx, const metis_adamw_tensor* const* ts, int count, const Coef& c) {
  static thread_local Table<CAP> tab;
  tab.c = c;
  tab.status = ctx->status;
  for (uint32_t r = 0; r < 10; ++r)
    tab.keys[r] = make_uint2((uint32_t)c.seed + r * 0x9E3779B9u, (uint32_t)(c.seed >> 32) + r * 0xBB67AE85u);
  // Chunks as large as leave every SM eight of them: the search for a chunk's tensor and the
  // tensor's addresses are paid once a chunk.
  int64_t elements = 0, chunks = 0;
  for (int i = 0; i < count; ++i) elements += ts[i]->n;
  tab.units = 1;
  while (tab.units < 16 && elements / (2 * tab.units * kUnit) >= 8 * (int64_t)ctx->sm_count) tab.units *= 2;
  const int64_t chunk = (int64_t)tab.units * kUnit;
  for (int i = 0; i < count; ++i) {
    const metis_adamw_tensor& x = *ts[i];
    tab.t[i] = Tensor{x.p, x.g, x.m, x.v, x.m_exponent, x.v_exponent, x.n};
    tab.id[i] = x.id;
    tab.first[i] = chunks;
    chunks += (x.n + chunk - 1) / chunk;
  }
  tab.count = count;
  tab.chunks = chunks;
  const int64_t grid = std::min<int64_t>(chunks, (int64_t)ctx->sm_count * (BITS == 32 ? 5 : 3));
  return launch_early(adamw_kernel<T, BITS, SR, CAP>, grid, kThreads, kRing<T, BITS, SR> ? sizeof(Ring<T>) : 0, ctx->stream, tab);
}

template <typename T, int BITS, bool SR>
cudaError_t launch_list(metis_ctx* ctx, const std::vector<const metis_adamw_tensor*>& ts, const Coef& c) {
  constexpr int kSmall = 48, kLarge = 400;
  for (size_t at = 0; at < ts.size();) {
    const int n = (int)std::min<size_t>(ts.size() - at, kLarge);
    const cudaError_t e = n <= kSmall ? launch_cap<T, BITS, SR, kSmall>(ctx, &ts[at], n, c)
                                      : launch_cap<T, BITS, SR, kLarge>(ctx, &ts[at], n, c);
    if (e != cudaSuccess) return e;
    at += n;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t launch_type(metis_ctx* ctx, const std::vector<const metis_adamw_tensor*>& ts, const Coef& c, int bits,
                        bool sr) {
  if (bits == 32) {
    // fp32 parameters with fp32 states are not rounded, so the rounding makes no difference
    if (sr && sizeof(T) == 2) return launch_list<T, 32, true>(ctx, ts, c);
    return launch_list<T, 32, false>(ctx, ts, c);
  }
  return sr ? launch_list<T, 8, true>(ctx, ts, c) : launch_list<T, 8, false>(ctx, ts, c);
}

}  // namespace

metis_status run_adamw(metis_ctx* ctx, const metis_adamw_tensor* tensors, int64_t count, const metis_adamw_params* q) {
  const Coef c{q->beta1, q->beta2, q->lr, q->weight_decay, q->eps, q->step, q->lr_dev, q->step_dev, q->seed};
  std::vector<const metis_adamw_tensor*> of[2];
  for (int64_t i = 0; i < count; ++i)
    if (tensors[i].n > 0) of[tensors[i].dtype == METIS_OUT_BF16].push_back(&tensors[i]);
  cudaError_t e = cudaSuccess;
  if (!of[0].empty()) e = launch_type<float>(ctx, of[0], c, q->state_bits, q->rounding == 1);
  if (e == cudaSuccess && !of[1].empty()) e = launch_type<__nv_bfloat16>(ctx, of[1], c, q->state_bits, q->rounding == 1);
  return check_cuda(ctx, e, "adamw launch");
}

}  // namespace metis
