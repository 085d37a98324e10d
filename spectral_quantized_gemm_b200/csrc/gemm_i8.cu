// Product of 8-bit integer matrices with a scale for each row of both operands:
//   C[i][j] = (sum_k A[i][k] B[j][k]) * sA[i] * sB[j]
// on the sm_100a tensor cores (tcgen05 kind::i8, int32 accumulators in tensor memory).  The
// sum is exact (K <= 131071 keeps it below 2^31); it is rounded to fp32 once, then
// multiplied by sA[i] and by sB[j], then rounded to the output type.
//
// gemm_i8_kernel: a cluster of S CTAs computes one 128 x BN tile, each CTA a share of K;
// the int32 sums are joined through distributed shared memory (the order of integer
// additions does not matter) and every CTA writes its part of the tile.
//   warp 0      TMA producer, 128-byte swizzled tiles of 128 K elements; zeros past the edges
//   warp 1      tensor-memory owner and MMA issuer (one thread)
//   warps 2..5  epilogue
// With few rows of A (tokens) the roles are swapped: B's rows (channels) take the 128
// lanes of the tile and the tokens its BN columns, so no lane idles.
// Every mbarrier wait is bounded; on expiry the CTA raises METIS_DEV_TIMEOUT, stops
// issuing work and exits after releasing its tensor memory.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "device_common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace metis {
namespace {

constexpr int kThreads = 192;
constexpr int kEpiThreads = 128;

struct Params {
  const float* sa;
  const float* sb;
  void* C;
  int64_t ldc;
  int64_t p, q;          // rows and columns of C
  int f32;
  int lane_tiles;        // 128-row blocks of the operand on the lanes
  int k_tiles;           // 128-element blocks of K
  uint32_t* status;
};

template <int BN>
struct Cfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN <= 64 ? 4 : 3;      // two CTAs fit an SM
  static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
  // staged sums: rows of the output, 4 words of padding so that 16-byte accesses of
  // consecutive rows fall on different banks
  static constexpr int STAGED = (BN + 4) * 128 > (128 + 4) * BN ? (BN + 4) * 128 * 4 : (128 + 4) * BN * 4;
  static constexpr int RING = STAGES * STAGE_BYTES;
  static constexpr size_t SMEM = (size_t)(RING > STAGED ? RING : STAGED) + 1024 + 256;
  static_assert(SMEM <= 116000, "two CTAs an SM");
};

__device__ __forceinline__ int4 load_cluster_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int BN, bool SWAP>
__global__ void __launch_bounds__(kThreads)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap map_lane, const __grid_constant__ CUtensorMap map_col,
                   const Params p) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (C::RING > C::STAGED ? C::RING : C::STAGED));
  uint64_t* full = bars;
  uint64_t* empty = bars + C::STAGES;
  uint64_t* done = bars + 2 * C::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = (int)tc::cluster_size();
  const int split = (int)tc::cluster_rank();
  const int tile = blockIdx.x / splits;
  const int lb = tile % p.lane_tiles, cb = tile / p.lane_tiles;
  const int s0 = (int)((int64_t)p.k_tiles * split / splits), s1 = (int)((int64_t)p.k_tiles * (split + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(done, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(&map_lane);
    tc::prefetch_tensormap(&map_col);
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int kk = s0; kk < s1; ++kk) {
        if (!tc::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
          *abort_flag = 1;
          raise_status(p.status, METIS_DEV_TIMEOUT);
          break;
        }
        uint8_t* sa = smem + stage * C::STAGE_BYTES;
        tc::mbar_expect_tx(&full[stage], C::STAGE_BYTES);
        tc::tma_load_2d(sa, &map_lane, &full[stage], kk * 128, lb * 128);
        tc::tma_load_2d(sa + C::A_BYTES, &map_col, &full[stage], kk * 128, cb * BN);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        ++issued;
      }
      // after a timeout too, no load is in flight when the block goes on
      for (int k = min(issued, C::STAGES); k > 0; --k) {
        if (--stage < 0) {
          stage = C::STAGES - 1;
          phase ^= 1u;
        }
        tc::mbar_wait(&full[stage], phase, nullptr);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      const uint32_t id = tc::idesc_i8(BN);
      for (int kk = s0; kk < s1; ++kk) {
        if (!tc::mbar_wait(&full[stage], phase, abort_flag)) {
          *abort_flag = 1;
          raise_status(p.status, METIS_DEV_TIMEOUT);
          break;
        }
        tc::tc_fence_after();
        const uint32_t sa = tc::smem_addr(smem + stage * C::STAGE_BYTES);
        const uint64_t ad = tc::sdesc_sw128(sa), bd = tc::sdesc_sw128(sa + C::A_BYTES);
#pragma unroll
        for (int j = 0; j < 4; ++j) tc::mma_i8(tmem, ad + 2 * j, bd + 2 * j, id, (kk != s0 || j) ? 1u : 0u);
        tc::tc_commit(&empty[stage]);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      tc::tc_commit(done);
      // every issued tensor-core operation ends before the memory is released
      if (!tc::mbar_wait(done, 0, nullptr)) {
        *abort_flag = 1;
        raise_status(p.status, METIS_DEV_TIMEOUT);
      }
    }
    __syncwarp();
  }
  // All loads have landed and all MMAs are done once every thread is here: the ring's
  // memory becomes the staging buffer.
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  int* staged = reinterpret_cast<int*>(smem);
  if (warp >= 2) {
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    constexpr int W = BN < 32 ? 16 : 32;
#pragma unroll
    for (int c = 0; c < BN; c += W) {
      float f[W];
      const uint32_t addr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c;
      if constexpr (W == 16) tc::tmem_load_16cols(addr, f); else tc::tmem_load_32cols(addr, f);
      tc::tmem_load_wait();
      if constexpr (SWAP) {
#pragma unroll
        for (int i = 0; i < W; ++i) staged[(c + i) * (128 + 4) + row] = __float_as_int(f[i]);
      } else {
#pragma unroll
        for (int i = 0; i < W; i += 4)
          *reinterpret_cast<int4*>(staged + row * (BN + 4) + c + i) =
              make_int4(__float_as_int(f[i]), __float_as_int(f[i + 1]), __float_as_int(f[i + 2]), __float_as_int(f[i + 3]));
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (splits > 1) tc::cluster_sync();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, C::TMEM_COLS);
  }
  // This CTA's part of the tile: runs of 8 columns of C, a 16-byte store of bf16 or two of fp32.
  {
    constexpr int ROWS = SWAP ? BN : 128, COLS = SWAP ? 128 : BN, RUNS = COLS / 8;
    const int64_t r0 = SWAP ? (int64_t)cb * BN : (int64_t)lb * 128, c0 = SWAP ? (int64_t)lb * 128 : (int64_t)cb * BN;
    const uint32_t mine = tc::smem_addr(staged);
    const int u1 = ROWS * RUNS * (split + 1) / splits;
    for (int u = ROWS * RUNS * split / splits + (int)threadIdx.x; u < u1; u += kThreads) {
      const int64_t i = r0 + u / RUNS, j = c0 + (u % RUNS) * 8;
      if (i >= p.p || j >= p.q) continue;
      const uint32_t off = (uint32_t)((u / RUNS) * (COLS + 4) + (u % RUNS) * 8) * 4u;
      int acc[8] = {};
      if (splits == 1) {
        const int4 a = *reinterpret_cast<const int4*>(smem + off), b = *reinterpret_cast<const int4*>(smem + off + 16);
        acc[0] = a.x; acc[1] = a.y; acc[2] = a.z; acc[3] = a.w;
        acc[4] = b.x; acc[5] = b.y; acc[6] = b.z; acc[7] = b.w;
      } else {
        for (int s = 0; s < splits; ++s) {
          const uint32_t from = tc::cluster_addr_u32(mine + off, (uint32_t)s);
          const int4 a = load_cluster_int4(from), b = load_cluster_int4(from + 16);
          acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
          acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
        }
      }
      const float sa = p.sa[i];
      const bool whole = j + 8 <= p.q;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (float)acc[e] * sa * (j + e < p.q ? p.sb[j + e] : 0.0f);
      if (p.f32) {
        float* dst = static_cast<float*>(p.C) + i * p.ldc + j;
        if (whole) {
          *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<float4*>(dst + 4) = make_float4(o[4], o[5], o[6], o[7]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (j + e < p.q) dst[e] = o[e];
        }
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.C) + i * p.ldc + j;
        if (whole) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 pr = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&pr);
          }
          *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (j + e < p.q) dst[e] = __float2bfloat16_rn(o[e]);
        }
      }
    }
  }
  if (splits > 1) tc::cluster_sync();   // no CTA leaves while its sums are still read
}

bool make_map_i8(CUtensorMap* map, const metis_int8* t, uint32_t box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)t->inner, (cuuint64_t)t->outer};
  const cuuint64_t strides[1] = {(cuuint64_t)t->ld};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, t->codes, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool SWAP>
metis_status launch_tile(metis_ctx* ctx, const metis_int8* A, const metis_int8* B, Params prm, int splits) {
  using C = Cfg<BN>;
  const metis_int8 *on_lanes = SWAP ? B : A, *on_cols = SWAP ? A : B;
  CUtensorMap ml, mc;
  if (!make_map_i8(&ml, on_lanes, 128) || !make_map_i8(&mc, on_cols, BN))
    return fail(ctx, METIS_ERR_CUDA, "cuTensorMapEncodeTiled failed for the int8 operands");
  const int64_t lane_tiles = (on_lanes->outer + 127) / 128, col_tiles = (on_cols->outer + BN - 1) / BN;
  if (lane_tiles * col_tiles * splits > INT32_MAX) return fail(ctx, METIS_ERR_SHAPE, "too many output tiles");
  prm.lane_tiles = (int)lane_tiles;
  auto kern = gemm_i8_kernel<BN, SWAP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return check_cuda(ctx, e, "cudaFuncSetAttribute(int8 gemm)");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(lane_tiles * col_tiles * splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = ctx->stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, ml, mc, prm);
  if (e != cudaSuccess) return check_cuda(ctx, e, "int8 gemm launch");
  count_launch();
  return METIS_OK;
}

}  // namespace

metis_status launch_gemm_i8(metis_ctx* ctx, const metis_int8* A, const metis_int8* B, void* C, int64_t ldc,
                            int32_t c_dtype) {
  Params prm{};
  prm.sa = A->scales;
  prm.sb = B->scales;
  prm.C = C;
  prm.ldc = ldc;
  prm.p = A->outer;
  prm.q = B->outer;
  prm.f32 = c_dtype == METIS_OUT_F32;
  prm.k_tiles = (int)((A->inner + 127) / 128);
  prm.status = ctx->status;
  return launch_tile<128, false>(ctx, A, B, prm, 1);
}

}  // namespace metis
