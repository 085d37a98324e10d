// Product of 8-bit integer matrices with a scale for each row of both operands:
//   C[i][j] = (sum_k A[i][k] B[j][k]) * sA[i] * sB[j]
// on the sm_100a tensor cores (tcgen05 kind::i8, int32 accumulators in tensor memory).  The
// sum is exact (K <= 131071 keeps it below 2^31); it is rounded to fp32 once, then
// multiplied by sA[i] and by sB[j], then rounded to the output type.
//
// gemm_i8_kernel: a cluster of S CTAs computes one tile of 128 rows of B (channels, on the
// lanes of tensor memory) by BN rows of A (tokens), each CTA a share of K.  Each CTA finishes
// some of the tokens: the others send it their int32 sums of these by asynchronous stores to its
// shared memory, whose bytes a barrier there counts, so nobody waits for a whole cluster (the
// order of integer additions does not matter).
//   warp 0      TMA producer, 128-byte swizzled tiles of 128 K elements; zeros past the edges
//   warp 1      tensor-memory owner and MMA issuer (one thread)
//   warps 2..5  epilogue
// Channels on the lanes suit few tokens (no lane idles) and let the staged sums be written
// and read without bank conflicts; at 512 x 768 x 2304 the other way round took 7.5 us where this
// one, with the same tile and no more changes, took 7.1.
//
// gemm_i8_pair_kernel: large products.  A cluster of two CTAs computes 256 x 256 tiles with
// cta_group::2 MMAs (each CTA loads 128 rows of A and 128 of B for every 128 K elements),
// persistent over the tiles, with two accumulators so that the epilogue of a tile runs
// under the MMAs of the next.  8192 x 4096 x 14336 takes 345 us in a row of others like it, at the power limit;
// a launch alone under the profiler took 325 with the tensor pipe busy 81% of the time.
//
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

constexpr int kThreads = 192, kMaxSplits = 8;

struct Params {
  const float* sa;
  const float* sb;
  void* C;
  int64_t ldc;
  int64_t p, q;          // rows and columns of C
  int f32;
  int lane_tiles;        // 128-row blocks of B
  int k_tiles;           // 128-element blocks of K
  int early;             // B may be read before the preceding kernel has ended
  uint32_t* status;
};

// A tile in S shares of K.  Tokens that a CTA finishes: a multiple of 4, so that four sums of a channel
// travel as 16 bytes.  They lie as [share][four tokens][channel][token] in its shared memory: a warp's
// store is 512 bytes in a row (with the channels apart it took twice as long).
__host__ __device__ constexpr int own_tokens(int bn, int splits) { return (bn / splits + (bn % splits != 0) + 3) / 4 * 4; }
constexpr int shared_sums(int bn) {   // bytes, for the S that needs most
  int most = 0;
  for (int s = 2; s <= kMaxSplits; ++s) {
    const int b = s * own_tokens(bn, s) * 128 * 4;
    most = b > most ? b : most;
  }
  return most;
}

// Many tiles, several CTAs an SM; up to one tile an SM; tiles in shares of K, each by a cluster (of two
// CTAs at least: the stores between them need a cluster launch).
enum Kind { kMany, kAlone, kShares };

template <int BN, Kind KIND>
struct Cfg {
  static constexpr bool SPLIT = KIND == kShares;
  static constexpr int A_BYTES = BN * 128;             // tokens
  static constexpr int B_BYTES = 128 * 128;            // channels
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TMEM_COLS = BN < 32 ? 32 : BN;
  // Stages of the ring.  A share with more than 16 tokens has its SM to itself: 5 (with quantizer: 40 x
  // 4096 x 4096 9.45 us with 4, 9.55 with 5, 10.2 with 7; 60 x 14336 x 4096 17.8, 17.1, 17.8).  A single
  // tile: 6 (32 x 4096 x 14336 18.2 us with 3, 15.7 with 6, 16.1 with 8).
  static constexpr int STAGES = KIND == kAlone ? 6 : SPLIT && BN > 16 ? 5 : SPLIT || BN == 32 ? 3 : 4;
  static constexpr int PER_SM = KIND == kAlone || (SPLIT && BN > 16) ? 1 : BN == 64 ? 2 : 3;
  static constexpr int PITCH = 128 + 4;                // words of a staged row of sums
  // One CTA a tile: the sums take the ring's place.  Several: a place of their own, which may be written
  // while this CTA still multiplies.
  static constexpr int STAGED = SPLIT ? shared_sums(BN) : BN * PITCH * 4;
  static constexpr int RING = SPLIT || STAGES * STAGE_BYTES > STAGED ? STAGES * STAGE_BYTES : STAGED;
  static constexpr size_t SMEM = (size_t)RING + (SPLIT ? STAGED : 0) + (128 + BN) * 4 + 1024 + 256;
  static_assert(STAGED % 16 == 0 && (SMEM + 1024) * PER_SM <= 233472, "CTAs an SM");
};

template <int BN, Kind KIND, typename OUT>
__global__ void __launch_bounds__(kThreads)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB, const Params p) {
  using C = Cfg<BN, KIND>;
  constexpr bool SPLIT = C::SPLIT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sb = reinterpret_cast<float*>(smem + C::RING + (SPLIT ? C::STAGED : 0));   // scales of the tile's channels and tokens
  float* sa = sb + 128;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sb + 128 + BN);
  uint64_t* full = bars;
  uint64_t* empty = bars + C::STAGES;
  uint64_t* done = bars + 2 * C::STAGES;
  uint64_t* received = done + 1;   // (SPLIT) the cluster's sums of this CTA's tokens are here
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = SPLIT ? (int)tc::cluster_size() : 1;
  const int split = SPLIT ? (int)tc::cluster_rank() : 0;
  const int tile = blockIdx.x / splits;
  const int lb = tile % p.lane_tiles, cb = tile / p.lane_tiles;
  const int s0 = (int)((int64_t)p.k_tiles * split / splits), s1 = (int)((int64_t)p.k_tiles * (split + 1) / splits);

  const int first = min(C::STAGES, s1 - s0);   // the first round of the ring
  // tokens of the tile, and this CTA's: own0 .. own1 - 1
  const int rows = (int)min((int64_t)BN, p.p - (int64_t)cb * BN), share = SPLIT ? own_tokens(BN, splits) : BN;
  const int own0 = min(rows, split * share), own1 = min(rows, own0 + share);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(done, 1);
    if (SPLIT) tc::mbar_init(received, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
    if (SPLIT) tc::mbar_expect_tx(received, (uint32_t)(splits * ((own1 - own0 + 3) & ~3) * 128 * 4));
    // the first loads leave before the other threads are ready; in a chain B's under the tail of the
    // preceding kernel
    if (!p.early) tc::grid_dependency_wait();
    for (int s = 0; s < first; ++s) {
      tc::mbar_expect_tx(&full[s], C::STAGE_BYTES);
      tc::tma_load_2d(smem + s * C::STAGE_BYTES + C::A_BYTES, &mapB, &full[s], (s0 + s) * 128, lb * 128);
      if (!p.early) tc::tma_load_2d(smem + s * C::STAGE_BYTES, &mapA, &full[s], (s0 + s) * 128, cb * BN);
    }
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, C::TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  if (SPLIT) tc::cluster_arrive_relaxed();   // this CTA's barrier is ready for the others' sums
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      if (p.early) {
        tc::grid_dependency_wait();
        for (int s = 0; s < first; ++s)
          tc::tma_load_2d(smem + s * C::STAGE_BYTES, &mapA, &full[s], (s0 + s) * 128, cb * BN);
      }
      int stage = first == C::STAGES ? 0 : first, issued = first;
      uint32_t phase = first == C::STAGES ? 1u : 0u;
      for (int kk = s0 + first; kk < s1; ++kk) {
        if (!tc::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
          *abort_flag = 1;
          raise_status(p.status, METIS_DEV_TIMEOUT);
          break;
        }
        uint8_t* at = smem + stage * C::STAGE_BYTES;
        tc::mbar_expect_tx(&full[stage], C::STAGE_BYTES);
        tc::tma_load_2d(at + C::A_BYTES, &mapB, &full[stage], kk * 128, lb * 128);
        tc::tma_load_2d(at, &mapA, &full[stage], kk * 128, cb * BN);
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
        const uint32_t at = tc::smem_addr(smem + stage * C::STAGE_BYTES);
        const uint64_t lanes = tc::sdesc_sw128(at + C::A_BYTES), cols = tc::sdesc_sw128(at);
#pragma unroll
        for (int j = 0; j < 4; ++j) tc::mma_i8(tmem, lanes + 2 * j, cols + 2 * j, id, (kk != s0 || j) ? 1u : 0u);
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
  } else {
    // the tile's scales, fetched while the sums are made
    const int t = (int)threadIdx.x - 64;
    const int64_t j = (int64_t)lb * 128 + t;
    if (!p.early) tc::grid_dependency_wait();
    sb[t] = j < p.q ? __ldcg(&p.sb[j]) : 0.0f;   // from L2: no cache of this SM can hold an older one
    if (p.early) tc::grid_dependency_wait();
    tc::grid_launch_dependents();
    if (t < BN) sa[t] = (int64_t)cb * BN + t < p.p ? p.sa[(int64_t)cb * BN + t] : 0.0f;
  }
  // All loads have landed and all MMAs are done once every thread is here.
  tc::tc_fence_before();
  __syncthreads();
  if (SPLIT) tc::cluster_wait();
  tc::tc_fence_after();
  int* staged = reinterpret_cast<int*>(smem + (SPLIT ? C::RING : 0));
  if (warp >= 2 && !(SPLIT && *abort_flag)) {
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    constexpr int W = BN < 32 ? 16 : 32;
    // (SPLIT) where the sums of the current tokens go: CTA 0's first
    const uint32_t here = tc::smem_addr(staged + split * share * 128 + row * 4);
    int owner = 0, left = share;
    uint32_t to = SPLIT ? tc::cluster_addr_u32(here, 0) : 0u, bar = SPLIT ? tc::cluster_addr_u32(tc::smem_addr(received), 0) : 0u;
#pragma unroll
    for (int c = 0; c < BN; c += W) {
      float f[W];
      const uint32_t addr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c;
      if constexpr (W == 16) tc::tmem_load_16cols(addr, f); else tc::tmem_load_32cols(addr, f);
      tc::tmem_load_wait();
      if constexpr (SPLIT) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
          if (c + i < rows)
            tc::store_async4(to, __float_as_uint(f[i]), __float_as_uint(f[i + 1]), __float_as_uint(f[i + 2]), __float_as_uint(f[i + 3]), bar);
          to += 128 * 16;
          if ((left -= 4) == 0) {                       // the next CTA's tokens
            left = share;
            ++owner;
            to = tc::cluster_addr_u32(here, (uint32_t)min(owner, splits - 1));
            bar = tc::cluster_addr_u32(tc::smem_addr(received), (uint32_t)min(owner, splits - 1));
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) staged[(c + i) * C::PITCH + row] = __float_as_int(f[i]);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, C::TMEM_COLS);
  }
  const int cols = (int)min((int64_t)128, p.q - (int64_t)lb * 128);
  OUT* const c0 = static_cast<OUT*>(p.C) + (int64_t)cb * BN * p.ldc + (int64_t)lb * 128;
  if (SPLIT && warp >= 2) {
    // This CTA's tokens, a thread a channel.  After a timeout too, the wait lasts until nothing more can
    // arrive here.
    const bool here = own1 == own0 || tc::mbar_wait_cluster(received, 0);
    if (!here && lane == 0) raise_status(p.status, METIS_DEV_TIMEOUT);
    const int t = (int)threadIdx.x - 64;
    const float sj = sb[t];
    for (int i = own0; here && t < cols && i < own1; i += 4) {
      int4 a = make_int4(0, 0, 0, 0);
      for (int s = 0; s < splits; ++s) {
        const int4 x = *reinterpret_cast<const int4*>(staged + (s * share + i - own0) * 128 + t * 4);
        a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
      }
      const int sums[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < own1) c0[(int64_t)(i + e) * p.ldc + t] = (OUT)((float)sums[e] * sa[i + e] * sj);
    }
  } else if (!SPLIT && warp >= 2) {
    // Runs of 8 columns of C, a 16-byte store of bf16 or two of fp32.  Kept small (one output type, not
    // unrolled): a CTA runs it once, and unrolled four times its instructions took 0.5 us longer to
    // come in than they saved.
    constexpr int RUNS = 128 / 8;
    for (int u = (int)threadIdx.x - 64; u < rows * RUNS; u += kThreads - 64) {
      const int i = u / RUNS, j = (u % RUNS) * 8;
      if (j >= cols) continue;
      const int* from = staged + i * C::PITCH + j;
      const int4 a = *reinterpret_cast<const int4*>(from), b = *reinterpret_cast<const int4*>(from + 4);
      const float si = sa[i];
      const float4 t0 = *reinterpret_cast<const float4*>(sb + j), t1 = *reinterpret_cast<const float4*>(sb + j + 4);
      const float o[8] = {(float)a.x * si * t0.x, (float)a.y * si * t0.y, (float)a.z * si * t0.z, (float)a.w * si * t0.w,
                          (float)b.x * si * t1.x, (float)b.y * si * t1.y, (float)b.z * si * t1.z, (float)b.w * si * t1.w};
      OUT* dst = c0 + (int64_t)i * p.ldc + j;
      if (j + 8 <= cols) {
        if constexpr (sizeof(OUT) == 4) {
          *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<float4*>(dst + 4) = make_float4(o[4], o[5], o[6], o[7]);
        } else {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 pr = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&pr);
          }
          *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (j + e < cols) dst[e] = (OUT)o[e];
      }
    }
  }
}

// ------------------------------------------------------------------ CTA-pair kernel
struct PairCfg {
  static constexpr int STAGE_BYTES = 2 * 128 * 128;
  static constexpr int STAGES = 6;
  static constexpr int EPI_WARPS = 8;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int BOX_BYTES = 4096;               // 32 rows x 128 bytes of the output, a warp's staging
  static constexpr size_t SMEM = (size_t)STAGES * STAGE_BYTES + EPI_WARPS * BOX_BYTES + 1024 + 256;
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct PairParams {
  const float* sa;
  const float* sb;
  int64_t p, q;
  void* C;
  int64_t ldc;
  int f32;
  int m_tiles, n_tiles, k_tiles;
  uint32_t* status;
};

// Columns of C that the TMA stores write: it clips at the matrix's edge in units of 16 bytes
// (measured: with 1333 bf16 columns it wrote 1336), so the odd last ones leave by plain stores.
inline __host__ __device__ int64_t whole_columns(int64_t q, int f32) { return f32 ? q & ~int64_t(3) : q & ~int64_t(7); }

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg::THREADS, 1)
    gemm_i8_pair_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                        const __grid_constant__ CUtensorMap mapC, const PairParams p) {
  using C = PairCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* epi = smem + C::STAGES * C::STAGE_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(epi + C::EPI_WARPS * C::BOX_BYTES);
  uint64_t* full = bars;                       // (even CTA) the pair's stage landed
  uint64_t* empty = bars + C::STAGES;          // the pair's MMAs are done with the stage
  uint64_t* acc_full = bars + 2 * C::STAGES;   // [2] this CTA's accumulator is complete
  uint64_t* acc_empty = acc_full + 2;          // [2] (even CTA) both CTAs have read theirs
  uint64_t* drain = acc_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], 2 * C::EPI_WARPS);
    }
    tc::mbar_init(drain, 1);
    *abort_flag = 0;
    tc::fence_barrier_init();
    tc::prefetch_tensormap(&mapA);
    tc::prefetch_tensormap(&mapB);
    tc::prefetch_tensormap(&mapC);
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tmem_slot, 512);
    tc::tmem_relinquish_pair();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();   // both CTAs' barriers exist before any cross-CTA arrival
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  tc::grid_dependency_wait();
  tc::grid_launch_dependents();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int num_tiles = p.m_tiles * p.n_tiles;

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    if (lane == 0) {
      const uint32_t full0 = tc::cluster_addr(&full[0], 0);
      int stage = 0;
      int64_t issued = 0;
      uint32_t phase = 0;
      for (int tile = pair; tile < num_tiles && !*abort_flag; tile += npairs) {
        const int arow = (tile % p.m_tiles) * 256 + (int)rank * 128;
        const int brow = (tile / p.m_tiles) * 256 + (int)rank * 128;
        for (int kk = 0; kk < p.k_tiles; ++kk) {
          if (!tc::mbar_wait(&empty[stage], phase ^ 1u, abort_flag)) {
            *abort_flag = 1;
            raise_status(p.status, METIS_DEV_TIMEOUT);
            break;
          }
          uint8_t* sa = smem + stage * C::STAGE_BYTES;
          const uint32_t fb = full0 + 8u * (uint32_t)stage;
          if (rank == 0) tc::mbar_expect_tx(&full[stage], 2 * C::STAGE_BYTES);
          tc::tma_load_2d_pair(sa, &mapA, fb, kk * 128, arow);
          tc::tma_load_2d_pair(sa + 128 * 128, &mapB, fb, kk * 128, brow);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          ++issued;
        }
      }
      // after a timeout too, no load of the pair is in flight past the last cluster barrier
      if (rank == 0)
        for (int k = (int)min(issued, (int64_t)C::STAGES); k > 0; --k) {
          if (--stage < 0) {
            stage = C::STAGES - 1;
            phase ^= 1u;
          }
          tc::mbar_wait(&full[stage], phase, nullptr, tc::kWaitLimitCycles / 8);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && rank == 0) {
      int stage = 0, it = 0;
      uint32_t phase = 0;
      const uint32_t id = tc::idesc_i8(256, 256);
      for (int tile = pair; tile < num_tiles && !*abort_flag; tile += npairs, ++it) {
        const int buf = it & 1;
        if (!tc::mbar_wait(&acc_empty[buf], ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag)) {
          *abort_flag = 1;
          raise_status(p.status, METIS_DEV_TIMEOUT);
          break;
        }
        tc::tc_fence_after();
        const uint32_t acc = tmem + (uint32_t)buf * 256u;
        for (int kk = 0; kk < p.k_tiles; ++kk) {
          if (!tc::mbar_wait(&full[stage], phase, abort_flag)) {
            *abort_flag = 1;
            raise_status(p.status, METIS_DEV_TIMEOUT);
            break;
          }
          tc::tc_fence_after();
          const uint32_t sa = tc::smem_addr(smem + stage * C::STAGE_BYTES);
          const uint64_t ad = tc::sdesc_sw128(sa), bd = tc::sdesc_sw128(sa + 128 * 128);
#pragma unroll
          for (int j = 0; j < 4; ++j) tc::mma_i8_pair(acc, ad + 2 * j, bd + 2 * j, id, (kk || j) ? 1u : 0u);
          tc::tc_commit_pair(&empty[stage], 0x3);
          if (++stage == C::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (*abort_flag) break;
        tc::tc_commit_pair(&acc_full[buf], 0x3);
      }
      // let every issued tensor-core operation finish before the memory is released
      tc::tc_commit_pair(drain, 0x1);
      tc::mbar_wait(drain, 0, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    // A warp takes 32 rows x 128 columns in pieces of one output box (128 bytes a row:
    // 64 bf16 or 32 fp32 columns): sums -> registers -> scaled into the swizzled box -> TMA
    // store, clipped at the matrix's edges.
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    const uint32_t empty_bar = tc::cluster_addr(&acc_empty[0], 0);
    uint8_t* box = epi + (warp - 2) * C::BOX_BYTES;
    const int swz = lane & 7;   // 16-byte chunk j of a box row r sits at position j ^ (r mod 8)
    int it = 0;
    for (int tile = pair; tile < num_tiles; tile += npairs, ++it) {
      const int buf = it & 1;
      const bool ok = __all_sync(0xffffffffu, tc::mbar_wait(&acc_full[buf], (uint32_t)(it >> 1) & 1u, abort_flag));
      if (!ok) {
        if (lane == 0) {
          *abort_flag = 1;
          raise_status(p.status, METIS_DEV_TIMEOUT);
        }
        break;
      }
      tc::tc_fence_after();
      const int y = (tile % p.m_tiles) * 256 + (int)rank * 128 + quarter * 32;
      const int x0 = (tile / p.m_tiles) * 256 + half * 128;
      const float sa = y + lane < p.p ? p.sa[y + lane] : 0.0f;
      const uint32_t acc = tmem + (uint32_t)buf * 256u + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * 128);
      const int last = (int)p.q - 1, whole = (int)whole_columns(p.q, p.f32);
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        float v[32];
        tc::tmem_load_32cols(acc + (uint32_t)c, v);
        tc::tmem_load_wait();
        if (c == 96) {
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_cluster(empty_bar + 8u * (uint32_t)buf);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = (float)__float_as_int(v[i]) * sa * p.sb[min(x0 + c + i, last)];
        if (whole <= last && x0 + c <= last && x0 + c + 32 > whole && y + lane < p.p) {
          const int64_t at = (int64_t)(y + lane) * p.ldc + x0 + c;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (x0 + c + i >= whole && x0 + c + i <= last) {
              if (p.f32) static_cast<float*>(p.C)[at + i] = v[i];
              else static_cast<__nv_bfloat16*>(p.C)[at + i] = __float2bfloat16_rn(v[i]);
            }
        }
        if (p.f32 || c % 64 == 0) {
          if (lane == 0) tc::bulk_wait_read_all();   // the last store has left the box
          __syncwarp();
        }
        if (p.f32) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(box + lane * 128 + ((j ^ swz) << 4)) =
                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 pr = __floats2bfloat162_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
              w[i] = *reinterpret_cast<const uint32_t*>(&pr);
            }
            *reinterpret_cast<uint4*>(box + lane * 128 + (((j + (c % 64) / 8) ^ swz) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (p.f32 || c % 64 == 32) {
          tc::fence_proxy_async();
          __syncwarp();
          const int x = x0 + (p.f32 ? c : c - 32);
          if (lane == 0 && x < whole && y < p.p) {
            tc::tma_store_2d(&mapC, box, x, y);
            tc::bulk_commit_group();
          }
        }
      }
    }
    if (lane == 0) tc::bulk_wait_all();   // stores complete before the boxes go away
    __syncwarp();
  }

  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();   // no cross-CTA access is outstanding past this point
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, 512);
  }
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

template <int BN, Kind KIND, typename OUT>
metis_status launch_tile(metis_ctx* ctx, const metis_int8* A, const metis_int8* B, Params prm, int splits, bool chained) {
  using C = Cfg<BN, KIND>;
  CUtensorMap ma, mb;
  if (!make_map_i8(&ma, A, BN) || !make_map_i8(&mb, B, 128))
    return fail(ctx, METIS_ERR_CUDA, "cuTensorMapEncodeTiled failed for the int8 operands");
  const int64_t lane_tiles = (prm.q + 127) / 128, col_tiles = (prm.p + BN - 1) / BN;
  const int64_t ctas = lane_tiles * col_tiles * splits;
  if (ctas > INT32_MAX) return fail(ctx, METIS_ERR_SHAPE, "too many output tiles");
  prm.lane_tiles = (int)lane_tiles;
  auto kern = gemm_i8_kernel<BN, KIND, OUT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return check_cuda(ctx, e, "cudaFuncSetAttribute(int8 gemm)");
  prm.early = chained;
  e = launch_early_cluster(kern, ctas, kThreads, C::SMEM, splits, ctx->stream, ma, mb, prm);
  if (e != cudaSuccess) return check_cuda(ctx, e, "int8 gemm launch");
  return METIS_OK;
}

bool make_map_out(CUtensorMap* map, const Params& prm) {
  const cuuint64_t dims[2] = {(cuuint64_t)whole_columns(prm.q, prm.f32), (cuuint64_t)prm.p};
  const cuuint64_t strides[1] = {(cuuint64_t)prm.ldc * (prm.f32 ? 4 : 2)};
  const cuuint32_t box[2] = {prm.f32 ? 32u : 64u, 32};
  const cuuint32_t estr[2] = {1, 1};
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  return enc(map, prm.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, prm.C, dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

metis_status launch_pair(metis_ctx* ctx, const metis_int8* A, const metis_int8* B, const Params& prm) {
  using C = PairCfg;
  CUtensorMap ma, mb, mc;
  if (!make_map_i8(&ma, A, 128) || !make_map_i8(&mb, B, 128) || !make_map_out(&mc, prm))
    return fail(ctx, METIS_ERR_CUDA, "cuTensorMapEncodeTiled failed for the int8 product");
  const int64_t m_tiles = (prm.p + 255) / 256, n_tiles = (prm.q + 255) / 256;
  if (m_tiles * n_tiles > INT32_MAX / 2) return fail(ctx, METIS_ERR_SHAPE, "too many output tiles");
  const PairParams pp{prm.sa, prm.sb, prm.p, prm.q, prm.C, prm.ldc, prm.f32, (int)m_tiles, (int)n_tiles, prm.k_tiles, prm.status};
  const cudaError_t e = cudaFuncSetAttribute(gemm_i8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return check_cuda(ctx, e, "cudaFuncSetAttribute(int8 gemm pair)");
  const int grid = 2 * (int)std::min<int64_t>(m_tiles * n_tiles, ctx->sm_count / 2);
  return check_cuda(ctx, launch_early(gemm_i8_pair_kernel, grid, C::THREADS, C::SMEM, ctx->stream, ma, mb, mc, pp),
                    "int8 gemm pair launch");
}

}  // namespace

metis_status launch_gemm_i8(metis_ctx* ctx, const metis_int8* A, const metis_int8* B, void* C, int64_t ldc,
                            int32_t c_dtype, bool chained) {
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
  const int bn = prm.p <= 16 ? 16 : prm.p <= 32 ? 32 : 64;
  const int64_t tiles = ((prm.q + 127) / 128) * ((prm.p + bn - 1) / bn);
  // Tile kernel or CTA pairs.  While the tiles of the former fit the SMs at once (two each) it is
  // ahead: 512 x 4096 x 4096 15.3 us against 18.5, 1024 x 1024 x 1024 6.0 against 9.2; with a
  // second wave it is behind: 2048 x 512 x 2048 11.2 against 9.9.  Up to 128 rows of A leave half
  // of a pair's tile empty.  A pair's stores need a whole 16 bytes of columns (a tensor map's extent may
  // not be 0), so a product by fewer stays with the tiles at any length.
  if (prm.p > 128 && tiles > 2 * ctx->sm_count && whole_columns(prm.q, prm.f32) > 0) return launch_pair(ctx, A, B, prm);
  // Shares of K.  Up to 16 tokens several CTAs share an SM, and more of them stream the weight faster
  // (1 x 4096 x 4096: 11.9 us in one share, 6.2 in eight; 1 x 768 x 2304: 3.8, 2.9 in six;
  // 1 x 4096 x 14336: 14.0, 11.8 in three, 14.8 in four, which no longer fit the SMs three to
  // each).  With 32 or 64 a CTA takes an SM to itself, and eight blocks of K each (40 x 4096 x
  // 4096: 12.6, 7.8 in four, 12.2 in six; 60 x 14336 x 4096: 35.9, 15.1 in four, 21.4 in six; 512 x
  // 2304 x 768: 8.6, 8.6 in two, 12.8 in three).
  const int64_t room = (bn == 16 ? ctx->sm_count * 27 / 10 : ctx->sm_count) / tiles;
  const int splits = (int)std::max<int64_t>(1, std::min<int64_t>({kMaxSplits, room, prm.k_tiles / (bn == 16 ? 1 : 8)}));
  // The deeper ring where a weight is read once, from HBM, by up to one CTA an SM.  Where several CTAs read
  // it from L2 it is no faster (256 x 4096 x 4096 15.1 us, 15.0 without; 512 x 768 x 2304 7.0, 6.7).
  const bool alone = bn > 16 && prm.p <= bn && splits == 1 && tiles <= ctx->sm_count && prm.k_tiles >= 8;
  auto launch = [&](auto zero) {
    using OUT = decltype(zero);
#define METIS_TILE(BN, KIND) launch_tile<BN, KIND, OUT>(ctx, A, B, prm, splits, chained)
    if (bn == 16) return splits > 1 ? METIS_TILE(16, kShares) : METIS_TILE(16, kMany);
    if (bn == 32) return splits > 1 ? METIS_TILE(32, kShares) : alone ? METIS_TILE(32, kAlone) : METIS_TILE(32, kMany);
    return splits > 1 ? METIS_TILE(64, kShares) : alone ? METIS_TILE(64, kAlone) : METIS_TILE(64, kMany);
#undef METIS_TILE
  };
  return prm.f32 ? launch(float{}) : launch(__nv_bfloat16{});
}

}  // namespace metis
