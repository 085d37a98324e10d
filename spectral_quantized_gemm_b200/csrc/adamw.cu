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

namespace metis {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 2048;          // elements a block handles at a time: 16 state blocks
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
  uint32_t* status;
  uint32_t id[CAP];           // random stream of each tensor
  int64_t first[CAP];         // first chunk of each tensor
  Tensor t[CAP];
};

// What a step needs of its coefficients, in fp32.
struct Step {
  float decay, size, rbc2, eps;
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
  s.t = (uint32_t)t;
  return s;
}

__device__ __forceinline__ float stepped(float p, float m, float v, const Step& s) {
  return p * s.decay - s.size * (m / (sqrtf(v) * s.rbc2 + s.eps));
}

// Four consecutive elements from i on of a tensor of n; the others read as 0.
template <typename T>
__device__ __forceinline__ void load4(const T* a, int64_t i, int64_t n, bool vec, float (&x)[4]) {
  if (vec && i + 4 <= n) {
    if constexpr (sizeof(T) == 4) {
      const float4 u = *reinterpret_cast<const float4*>(a + i);
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(a + i);
      x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xFFFF0000u);
      x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = i + j < n ? (float)a[i + j] : 0.0f;
  }
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

// A code's magnitude is the fp64 number with bits code << 49 (exponent field code / 8, so
// that gradual underflow is the format's own) times 2^(1022 + E - 127 - octaves + 1).
__device__ __forceinline__ double decode(uint32_t code, double scale) {
  return __hiloint2double((int)(code << 17), 0) * power2(1000) * scale;
}
__device__ __forceinline__ double decode_scale(int top, int octaves) { return power2(22 + top - octaves + 1); }

// The code of a finite x >= 0 from t = x / u.  From 8 on, 3 mantissa bits are kept by an integer
// addition to the fp64 number (its exponent and upper mantissa bits count the codes); below
// 8 the grid's step is 1.
template <bool SR>
__device__ __forceinline__ uint32_t encode(double x, double per_unit, uint32_t field, uint32_t most) {
  const double t = x * per_unit;
  if (t < 8.0)
    return (uint32_t)(SR ? __double2int_rd(t + ((double)field + 0.5) * (1.0 / 65536.0)) : __double2int_rn(t));
  const unsigned long long b = (unsigned long long)__double_as_longlong(t);
  unsigned long long r;
  if (SR)
    r = ((unsigned long long)field << 33) + (1ull << 32);                 // (field + 1/2) 2^-16 of a step
  else
    r = ((1ull << 48) - 1) + ((b >> 49) & 1);                             // nearest, ties to even
  return min((uint32_t)((b + r) >> 49) - (1026u * 8u - 8u), most);        // 8.0 has the exponent field 1026
}
__device__ __forceinline__ double units(int top, int octaves) { return power2(octaves + 2 - top); }

__device__ __forceinline__ int exponent_field(double x) { return (__double2hiint(x) >> 20) & 0x7FF; }

// Exponent byte - 127 of a block from the largest fp64 exponent field of its elements
// (0x7FF, a NaN or an infinity, left out by the caller).
__device__ __forceinline__ int block_top(int field) { return min(max(field - 1023, -111), 127); }

template <typename T, int BITS, bool SR, int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<CAP> tab) {
  __shared__ Step sh;
  if (threadIdx.x == 0) sh = make_step(tab.c);
  __syncthreads();
  const Step s = sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  bool bad = false;
  for (int64_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    int lo = 0, hi = tab.count - 1;   // the last tensor whose first chunk is not beyond this one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.first[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    const Tensor& t = tab.t[lo];
    const int64_t n = t.n;
    const int64_t base = (chunk - tab.first[lo]) * kChunk;
    T* p = static_cast<T*>(t.p);
    const T* g = static_cast<const T*>(t.g);
    const uintptr_t mask = sizeof(T) == 4 ? 15u : 7u;
    const bool vec_p = (reinterpret_cast<uintptr_t>(p) & mask) == 0, vec_g = (reinterpret_cast<uintptr_t>(g) & mask) == 0;
    if constexpr (BITS == 32) {
      float* m = static_cast<float*>(t.m);
      float* v = static_cast<float*>(t.v);
      const bool vec_s = ((reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(v)) & 15u) == 0;
      const float b1 = (float)tab.c.b1, b2 = (float)tab.c.b2;
      const float a1 = (float)(1.0 - tab.c.b1), a2 = (float)(1.0 - tab.c.b2);
#pragma unroll
      for (int u = 0; u < kChunk / (kThreads * 4); ++u) {
        const int64_t i = base + (int64_t)(u * kThreads + threadIdx.x) * 4;
        if (i >= n) continue;
        float xp[4], xg[4], xm[4], xv[4];
        load4(p, i, n, vec_p, xp);
        load4(g, i, n, vec_g, xg);
        load4(m, i, n, vec_s, xm);
        load4(v, i, n, vec_s, xv);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bad |= !isfinite(xg[j]);
          xm[j] = fmaf(b1, xm[j], a1 * xg[j]);
          xv[j] = fmaf(b2, xv[j], a2 * (xg[j] * xg[j]));
          xp[j] = stepped(xp[j], xm[j], xv[j], s);
        }
        store4(m, i, n, vec_s, xm);
        store4(v, i, n, vec_s, xv);
        if constexpr (sizeof(T) == 4) {
          store4(p, i, n, vec_p, xp);
        } else {
          Words4 w{};
          if (SR) w = stream_call(tab.c.seed, stream_tag(tab.id[lo], kPurposeState, 1), s.t, (uint64_t)i >> 2);
          store4(p, i, n, vec_p, xp, SR, w);
        }
      }
    } else {
      uint8_t* m = static_cast<uint8_t*>(t.m);
      uint8_t* v = static_cast<uint8_t*>(t.v);
      const bool vec_s = ((reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(v)) & 3u) == 0;
      const double b1 = tab.c.b1, b2 = tab.c.b2;
#pragma unroll
      for (int u = 0; u < kChunk / (kThreads * 4); ++u) {
        // a warp takes one state block
        const int64_t i0 = base + (int64_t)(u * (kThreads / 32) + warp) * kStateBlock;
        if (i0 >= n) break;
        const int64_t i = i0 + lane * 4, blk = i0 / kStateBlock;
        float xp[4], xg[4];
        load4(p, i, n, vec_p, xp);
        load4(g, i, n, vec_g, xg);
        const uint32_t cm = load_codes(m, i, n, vec_s), cv = load_codes(v, i, n, vec_s);
        const double dm = decode_scale((int)t.me[blk] - 127, kMOctaves), dv = decode_scale((int)t.ve[blk] - 127, kVOctaves);
        double ym[4], yv[4];
        int fm = 0, fv = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t c = (cm >> (8 * j)) & 255u;
          const double old = decode(c & 127u, dm), gd = (double)xg[j];
          bad |= !isfinite(xg[j]);
          ym[j] = __dadd_rn(__dmul_rn(b1, c > 127u ? -old : old), __dmul_rn(1.0 - b1, gd));
          yv[j] = __dadd_rn(__dmul_rn(b2, decode((cv >> (8 * j)) & 255u, dv)), __dmul_rn(1.0 - b2, __dmul_rn(gd, gd)));
          const int em = exponent_field(ym[j]), ev = exponent_field(yv[j]);
          if (em != 0x7FF) fm = max(fm, em);
          if (ev != 0x7FF) fv = max(fv, ev);
          xp[j] = stepped(xp[j], (float)ym[j], (float)yv[j], s);
        }
        const int tm = block_top(__reduce_max_sync(0xffffffffu, fm)), tv = block_top(__reduce_max_sync(0xffffffffu, fv));
        const double sm = units(tm, kMOctaves), sv = units(tv, kVOctaves);
        Words4 w{};
        if (SR) w = stream_call(tab.c.seed, stream_tag(tab.id[lo], kPurposeState, 0), s.t, (uint64_t)i >> 2);
        uint32_t om = 0, ov = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t c = encode<SR>(fabs(ym[j]), sm, w.w[j] & 0xFFFFu, 127u);
          if (c && ym[j] < 0.0) c |= 128u;
          uint32_t e = max(encode<SR>(yv[j], sv, w.w[j] >> 16, 255u), yv[j] > 0.0 ? 1u : 0u);
          // an element whose gradient was not finite (its parameter is NaN now) restarts from zero
          if (exponent_field(ym[j]) == 0x7FF || exponent_field(yv[j]) == 0x7FF) c = e = 0;
          om |= c << (8 * j);
          ov |= e << (8 * j);
        }
        store_codes(m, i, n, vec_s, om);
        store_codes(v, i, n, vec_s, ov);
        if (lane == 0) {
          t.me[blk] = (uint8_t)(tm + 127);
          t.ve[blk] = (uint8_t)(tv + 127);
        }
        if constexpr (sizeof(T) == 4) {
          store4(p, i, n, vec_p, xp);
        } else {
          Words4 wp{};
          if (SR) wp = stream_call(tab.c.seed, stream_tag(tab.id[lo], kPurposeState, 1), s.t, (uint64_t)i >> 2);
          store4(p, i, n, vec_p, xp, SR, wp);
        }
      }
    }
  }
  if (bad) raise_status(tab.status, METIS_DEV_NONFINITE);
}

template <typename T, int BITS, bool SR, int CAP>
cudaError_t launch_cap(metis_ctx* ctx, const metis_adamw_tensor* const* ts, int count, const Coef& c) {
  static thread_local Table<CAP> tab;
  tab.c = c;
  tab.status = ctx->status;
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    const metis_adamw_tensor& x = *ts[i];
    tab.t[i] = Tensor{x.p, x.g, x.m, x.v, x.m_exponent, x.v_exponent, x.n};
    tab.id[i] = x.id;
    tab.first[i] = chunks;
    chunks += (x.n + kChunk - 1) / kChunk;
  }
  tab.count = count;
  tab.chunks = chunks;
  const int64_t grid = std::min<int64_t>(chunks, (int64_t)ctx->sm_count * 8);
  adamw_kernel<T, BITS, SR, CAP><<<(unsigned)grid, kThreads, 0, ctx->stream>>>(tab);
  count_launch();
  return cudaGetLastError();
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
