// The adapter's products of the microscaled layer on the tensor cores:
//
//   down   S[M, r]  = Z[M, L] R                T = X' A^T (R = A^T), U = dY B (R = B)
//   outer  G[C, r]  = Q[M, C]^T P[M, r]        dA^T from X' and s U, dB from dY and T
//
// Each reads a large bf16 matrix once and is bound by that read (r <= 128): T of
// 8192 x 3584, r = 64, 16.6 us, dA and dB of 8192 x 4096 each 27.5 us, 0.78 of the
// copy rate.  S leaves in bf16 because it is an operand of the next product's
// tensor cores: a rounding of half a step, 2^-8, of each of its elements.  A
// CTA sums a tile of 128 rows (tokens, or columns of Q) x r in tensor memory,
// operands by TMA: Z and A are K-major; where the contraction runs over a
// matrix's rows (Q, P, B) a tile of 64 rows x 64 columns lands as an MN-major
// operand and the MMA transposes it (no transposed copy is made).  A cluster
// splits the contraction over 2^log_splits CTAs, so that few rows still occupy
// the GPU, and adds the partial sums through distributed shared memory in rank
// order: one launch, no workspace, the same bits every time.
//
//  * warp 0: TMA (a stage: 64 of the contraction, 16 KB + 2 to 16 KB), as many
//    stages as fit, since the bytes in flight are what the read's rate needs:
//    with three stages a CTA took 0.33 us a stage, 54 GB/s;
//  * warp 1: tcgen05.mma kind::f16, M = 128, N = r (at least 16);
//  * warps 2-5: cluster reduction, rounding, stores.
//
// The tensor core truncates the sum that it adds to, so a contraction of n MMAs
// loses up to n half steps of it where all terms have one sign (8.4 M tokens: 65536 MMAs,
// dA and dB 0.5 % too small, more than their rounding).  A CTA's contraction is cut in
// runs of kRun stages (2048 MMAs, 2^-12 at most); warps 2-5 add up the runs, rounding
// to nearest, in columns of their own.
// Every wait is bounded (QLORA_ERR_TIMEOUT).

#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "gemm.h"
#include "mx.h"
#include "mx_gemm.cuh"
#include "mx_mma.cuh"
#include "draw.cuh"

namespace qnf4 {
namespace skinny {

using mx::elect_one;

constexpr int NUM_THREADS = 192;
constexpr int kMaxStages = 10;
constexpr int kRun = 512;                          // stages of a run, a power of two
constexpr int A_BYTES = 128 * 64 * 2;

// One product of a launch (an outer launch has up to two).
struct Problem {
  int rows;                 // tokens (down) or columns of Q (outer)
  int tiles;                // 128-row tiles
  const float* row_scale;   // down: pad[m] is divided by row_scale[m] (or null)
  __nv_bfloat16* pad;       // down: [rows, RP] = RNbf16(s S / row_scale), zero beyond r
  __nv_bfloat16* out;       // down: RNbf16(S) [rows, r] or null; outer: RNbf16(s G), [rows, r] or
  int transposed;           // [r, rows] (transposed)
  float s;
};
struct Args {
  Problem p[2];
  int L;                    // contraction length
  int r, N, RP;             // rank; MMA N (a power of two, 16 to 128); padded width
  int log_splits;
  int ns, b_bytes;          // stages and the bytes of B in one
  int wait_first;           // read nothing before the kernel before this one has ended
  int* status;
};

// Shared memory: this, then ns stages of A and B, 1024-byte aligned; the
// reduction's partial sums (N * 512 bytes) take the stages' place.
struct Head {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full, acc_empty;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Head) <= 1024, "stages begin at 1024");

// Two results of a row, columns col and col + 1.
template <bool OUTER>
__device__ __forceinline__ void store2(const Args& g, const Problem& p, const float* v, int row, int col) {
  if (row >= p.rows) return;
  if (OUTER) {
    if (col >= g.r) return;
    if (p.transposed) {
      p.out[(int64_t)col * p.rows + row] = __float2bfloat16_rn(__fmul_rn(p.s, v[0]));
      p.out[(int64_t)(col + 1) * p.rows + row] = __float2bfloat16_rn(__fmul_rn(p.s, v[1]));
    } else {
      *reinterpret_cast<uint32_t*>(p.out + (int64_t)row * g.r + col) =
          pack_bf16x2(__fmul_rn(p.s, v[0]), __fmul_rn(p.s, v[1]));
    }
  } else {
    float a = __fmul_rn(p.s, v[0]), b = __fmul_rn(p.s, v[1]);
    if (p.row_scale) {
      const float d = p.row_scale[row];
      a = __fdiv_rn(a, d);
      b = __fdiv_rn(b, d);
    }
    if (p.pad && col < g.RP) *reinterpret_cast<uint32_t*>(p.pad + (int64_t)row * g.RP + col) = pack_bf16x2(a, b);
    if (p.out && col < g.r) *reinterpret_cast<uint32_t*>(p.out + (int64_t)row * g.r + col) = pack_bf16x2(v[0], v[1]);
  }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Eight, columns col .. col + 7 (col a multiple of 8, like r).
template <bool OUTER>
__device__ __forceinline__ void store8(const Args& g, const Problem& p, const float* v, int row, int col) {
  if (row >= p.rows) return;
  if (OUTER && p.transposed) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) store2<OUTER>(g, p, v + j, row, col + j);
    return;
  }
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(p.s, v[j]);
  if (OUTER) {
    if (col < g.r) *reinterpret_cast<uint4*>(p.out + (int64_t)row * g.r + col) = pack8(f);
    return;
  }
  if (p.row_scale) {
    const float d = p.row_scale[row];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __fdiv_rn(f[j], d);
  }
  if (p.pad && col < g.RP) *reinterpret_cast<uint4*>(p.pad + (int64_t)row * g.RP + col) = pack8(f);
  if (p.out && col < g.r) *reinterpret_cast<uint4*>(p.out + (int64_t)row * g.r + col) = pack8(v);
}

// OUTER: both operands MN-major; RT (down): R [L, r] is.  LONG: several runs (in one
// kernel with the others, T and U of a backward each took 0.5 us more).
template <bool OUTER, bool RT, bool LONG>
__global__ void __launch_bounds__(NUM_THREADS, 2)
k_mx_skinny(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_b0,
            const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b1,
            const __grid_constant__ Args g) {
  constexpr uint32_t kCols = LONG ? 256 : 128;     // tensor-memory columns
  extern __shared__ uint8_t smem_raw[];
  grid_launch_dependents();
  Head& S = *smem_align1024<Head>(smem_raw);
  uint8_t* stages = reinterpret_cast<uint8_t*>(&S) + 1024;
  const int NS = g.ns, stage_bytes = A_BYTES + g.b_bytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ls = g.log_splits, splits = 1 << ls;
  const int rank = (int)cluster_ctarank();
  int tile = (int)(blockIdx.x >> ls);
  const bool second = tile >= g.p[0].tiles;
  const Problem& p = g.p[second ? 1 : 0];
  if (second) tile -= g.p[0].tiles;
  const CUtensorMap* tm_a = second ? &tm_a1 : &tm_a0;
  const CUtensorMap* tm_b = second ? &tm_b1 : &tm_b0;
  const int row0 = tile * 128;
  const int nk_all = (g.L + 63) / 64;
  const int k0 = (int)(((int64_t)nk_all * rank) >> ls), k1 = (int)(((int64_t)nk_all * (rank + 1)) >> ls);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.acc_empty, 4);
    S.abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, kCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(tm_a);
    tma_prefetch_desc(tm_b);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  volatile int* abort = &S.abort;
  const int runs = LONG ? (k1 - k0 + kRun - 1) / kRun : 1;
  const int quad = warp & 3;
  const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16);
  // 16 columns of the accumulator, with the runs before it
  auto sums16 = [&](int c, bool more, float* v) {
    tmem_ld16(taddr + c, reinterpret_cast<uint32_t*>(v));
    if (LONG && more) {
      float w[16];
      tmem_ld16(taddr + 128 + c, reinterpret_cast<uint32_t*>(w));
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __fadd_rn(v[j], w[j]);
    } else {
      tmem_wait_ld();
    }
  };
  if (g.wait_first) grid_dependency_wait();        // in every warp: a bounded wait begins with the work

  if (warp == 0) {
    if (elect_one()) {
      int s = 0, i = k0;
      uint32_t ph = 0;
      for (; i < k1; ++i) {
        if (!mbar_wait(&S.empty[s], ph ^ 1, abort, g.status)) break;
        mbar_arrive_expect_tx(&S.full[s], stage_bytes);
        uint8_t* a = stages + s * stage_bytes;
        uint8_t* b = a + A_BYTES;
        if (OUTER) {
          tma_load_2d(a, tm_a, &S.full[s], row0, i * 64);
          tma_load_2d(a + 8192, tm_a, &S.full[s], row0 + 64, i * 64);
        } else {
          tma_load_2d(a, tm_a, &S.full[s], i * 64, row0);
          if (!RT) tma_load_2d(b, tm_b, &S.full[s], i * 64, 0);
        }
        if (OUTER || RT)
          for (int j = 0; j * 8192 < g.b_bytes; ++j) tma_load_2d(b + j * 8192, tm_b, &S.full[s], j * 64, i * 64);
        if (++s == NS) { s = 0; ph ^= 1; }
      }
      if (*abort) {                                // a wait gave up: let the copies in flight land
        const int n = i - k0;
        for (int j = max(0, n - NS); j < n; ++j) mx::drain_wait(&S.full[j % NS], (j / NS) & 1, g.status);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16_f32(128, 16) + ((uint32_t)((g.N - 16) >> 3) << 17) +
                             (OUTER ? 1u << 15 : 0u) | (OUTER || RT ? 1u << 16 : 0u);
      int s = 0;
      uint32_t ph = 0;
      for (int i = k0; i < k1; ++i) {
        const int at = LONG ? (i - k0) & (kRun - 1) : i - k0;      // stage of the run
        if (LONG && at == 0 && i > k0) {
          mma_commit(&S.acc_full);
          if (!mbar_wait(&S.acc_empty, ((i - k0) / kRun - 1) & 1, abort, g.status)) break;
        }
        if (!mbar_wait(&S.full[s], ph, abort, g.status)) break;
        tc_fence_after();
        const uint32_t aa = smem_u32(stages + s * stage_bytes), bb = aa + A_BYTES;
        const uint64_t a = OUTER ? mx::mn_desc(aa, 8192) : sw128_kmajor_desc(aa);
        const uint64_t b = OUTER || RT ? mx::mn_desc(bb, 8192) : sw128_kmajor_desc(bb);
        constexpr uint32_t kRows = 2048 / 16, kElems = 32 / 16;  // 16 rows, or 16 elements of a row
#pragma unroll
        for (int q = 0; q < 4; ++q)
          mma_ss(tmem, a + (OUTER ? kRows : kElems) * q, b + (OUTER || RT ? kRows : kElems) * q, idesc,
                 (at > 0 || q > 0) ? 1u : 0u);
        mma_commit(&S.empty[s]);
        if (++s == NS) { s = 0; ph ^= 1; }
      }
      mma_commit(&S.acc_full);
      mbar_wait(&S.acc_full, (runs - 1) & 1, abort, g.status);
    }
  } else {
    for (int j = 0; LONG && j + 1 < runs && mbar_wait(&S.acc_full, j & 1, abort, g.status); ++j) {
      __syncwarp();
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < g.N; c += 16) {
        float v[16];
        sums16(c, j > 0, v);
        tmem_st16(taddr + 128 + c, reinterpret_cast<const uint32_t*>(v));
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.acc_empty);
    }
    mbar_wait(&S.acc_full, (runs - 1) & 1, abort, g.status);
    // as a dependent of the quantisation (whose row scales may be read below) this
    // grid does not end before that one
    grid_dependency_wait();
  }
  __syncwarp();
  const int at = quad * 32 + lane, row = row0 + at;
  if (ls == 0) {
    if (warp >= 2) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < g.N; c += 16) {
        float v[16];
        sums16(c, runs > 1, v);
        store8<OUTER>(g, p, v, row, c);
        store8<OUTER>(g, p, v + 8, row, c + 8);
      }
    }
  } else {
    cluster_sync();                                // every rank is done with its stages
    const int cs = g.N >> ls, lcs = __ffs(cs) - 1; // columns each rank adds up (a power of two)
    float* part = reinterpret_cast<float*>(stages);  // [splits][cs][128]
    if (warp >= 2) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < g.N; c += 16) {
        float v[16];
        sums16(c, runs > 1, v);
        const uint32_t mine = smem_u32(part + rank * cs * 128 + at);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          mx::st_cluster_f32(mapa_shared(mine + (uint32_t)(((c + j) & (cs - 1)) * 512), (c + j) >> lcs),
                             v[j]);
      }
    }
    cluster_sync();                                // the partial sums have arrived
    if (warp >= 2) {
      const float* b = part + at;
      if (cs >= 8) {
#pragma unroll 1
        for (int c = 0; c < cs; c += 8) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = b[(c + j) * 128];
          for (int z = 1; z < splits; ++z)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(v[j], b[(z * cs + c + j) * 128]);
          store8<OUTER>(g, p, v, row, rank * cs + c);
        }
      } else {
        for (int c = 0; c < cs; c += 2) {          // 2 or 4 columns
          float v[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            v[j] = b[(c + j) * 128];
            for (int z = 1; z < splits; ++z) v[j] = __fadd_rn(v[j], b[(z * cs + c + j) * 128]);
          }
          store2<OUTER>(g, p, v, row, rank * cs + c);
        }
      }
    }
  }
  if (!OUTER && warp >= 2 && rank == 0 && p.pad && row < p.rows)
    for (int c = g.N; c < g.RP; c += 8) *reinterpret_cast<uint4*>(p.pad + (int64_t)row * g.RP + c) = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// Ranks of a cluster and stages: up to one CTA an SM, of at least four stages
// each, with all of its shared memory; with more tiles than SMs two CTAs share
// one.  8192 x 4096, r = 64 (64 tiles): 17 us with 2 ranks and 8 stages against
// 29 us unsplit and 20.5 us with 4 ranks, two CTAs an SM of 3 stages.
static void shape(Args& g, int num_sms) {
  const int tiles = g.p[0].tiles + g.p[1].tiles, nk = (g.L + 63) / 64;
  int ls = 0;
  while (ls < 3 && (tiles << (ls + 1)) <= num_sms && (nk >> (ls + 1)) >= 4) ++ls;
  g.log_splits = ls;
  const int budget = ((tiles << ls) > num_sms ? 110 : 224) * 1024 - 2048;
  g.ns = std::min(kMaxStages, budget / (A_BYTES + g.b_bytes));
}

template <bool OUTER, bool RT, bool LONG>
static int launch_kernel(const CUtensorMap& a0, const CUtensorMap& b0, const CUtensorMap& a1, const CUtensorMap& b1,
                  const Args& g, bool beside, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_devs{0};
  set_smem_attr_once(k_mx_skinny<OUTER, RT, LONG>, 224 * 1024, attr_devs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(g.p[0].tiles + g.p[1].tiles) << g.log_splits, 1, 1);
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = 2048 + (size_t)g.ns * (A_BYTES + g.b_bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1u << g.log_splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_mx_skinny<OUTER, RT, LONG>, a0, b0, a1, b1, g) == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

template <bool OUTER, bool RT>
static int launch(const CUtensorMap& a0, const CUtensorMap& b0, const CUtensorMap& a1, const CUtensorMap& b1,
                  const Args& g, bool beside, cudaStream_t s) {
  const int nk = (g.L + 63) / 64;                  // a rank has at most this / 2^log_splits, rounded up
  return (nk + (1 << g.log_splits) - 1) >> g.log_splits > kRun ? launch_kernel<OUTER, RT, true>(a0, b0, a1, b1, g, beside, s)
                                                               : launch_kernel<OUTER, RT, false>(a0, b0, a1, b1, g, beside, s);
}

}  // namespace skinny

int launch_mx_down(const void* Z, const void* R, bool r_rows, int M, int L, int r, int RP, float s,
                   const float* row_scale, void* pad, void* out, After after, int* status, cudaStream_t st, int num_sms) {
  using namespace skinny;
  Args g{};
  g.L = L;
  g.r = r;
  g.N = std::max(r, 16);
  g.RP = RP;
  g.status = status;
  g.p[0] = Problem{M, (M + 127) / 128, row_scale, (__nv_bfloat16*)pad, (__nv_bfloat16*)out, 0, s};
  g.b_bytes = r_rows ? (g.N + 63) / 64 * 8192 : g.N * 128;
  g.wait_first = after == After::kWaits;
  shape(g, num_sms);
  CUtensorMap a, b;
  if (!make_tmap_2d_bf16(&a, Z, L, M, L, 64, 128) ||
      !(r_rows ? make_tmap_2d_bf16(&b, R, r, L, r, 64, 64) : make_tmap_2d_bf16(&b, R, L, r, L, 64, g.N)))
    return QLORA_ERR_CUDA;
  const bool beside = after != After::kEnds;
  return r_rows ? launch<false, true>(a, b, a, b, g, beside, st) : launch<false, false>(a, b, a, b, g, beside, st);
}

int launch_mx_outer(const void* Xd, int K, const void* sU, int ldu, void* dA, const void* dY, int N, const void* T,
                    float s, void* dB, int M, int r, int* status, cudaStream_t st, int num_sms) {
  using namespace skinny;
  Args g{};
  g.L = M;
  g.r = r;
  g.N = std::max(r, 16);
  g.status = status;
  g.p[0] = Problem{K, (K + 127) / 128, nullptr, nullptr, (__nv_bfloat16*)dA, 1, 1.0f};
  g.p[1] = Problem{N, (N + 127) / 128, nullptr, nullptr, (__nv_bfloat16*)dB, 0, s};
  g.b_bytes = (g.N + 63) / 64 * 8192;
  g.wait_first = 1;
  shape(g, num_sms);
  CUtensorMap a0, b0, a1, b1;
  if (!make_tmap_2d_bf16(&a0, Xd, K, M, K, 64, 64) || !make_tmap_2d_bf16(&b0, sU, r, M, ldu, 64, 64) ||
      !make_tmap_2d_bf16(&a1, dY, N, M, N, 64, 64) || !make_tmap_2d_bf16(&b1, T, r, M, r, 64, 64))
    return QLORA_ERR_CUDA;
  return launch<true, false>(a0, b0, a1, b1, g, true, st);
}

// ===========================================================================
// At[K, RP] = A[r, K]^T, zero beyond r, for the paired-SM GEMM and the masked term
// of dX: a CTA 64 columns of A through shared memory, 16-byte words of global
// memory on both sides.
// ===========================================================================
__global__ void __launch_bounds__(256)
k_mx_transpose(const __nv_bfloat16* __restrict__ A, int r, int K, int RP, __nv_bfloat16* __restrict__ At) {
  __shared__ uint16_t tile[64][130];               // [column of A][row of A]
  grid_launch_dependents();
  const int tid = threadIdx.x, k0 = blockIdx.x * 64;
  for (int i = tid; i < RP * 8; i += 256) {
    const int j = i >> 3, k = 8 * (i & 7);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (j < r && k0 + k < K) v = *reinterpret_cast<const uint4*>(A + (int64_t)j * K + k0 + k);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[k + e][j] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
  __syncthreads();
  for (int i = tid; i < 64 * (RP / 8); i += 256) {
    const int k = i / (RP / 8), j = 8 * (i % (RP / 8));
    if (k0 + k >= K) continue;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = tile[k][j + 2 * e] | (uint32_t)tile[k][j + 2 * e + 1] << 16;
    *reinterpret_cast<uint4*>(At + (int64_t)(k0 + k) * RP + j) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

void launch_mx_transpose(const void* A, int r, int K, int RP, void* At, cudaStream_t s) {
  k_mx_transpose<<<(K + 63) / 64, 256, 0, s>>>((const __nv_bfloat16*)A, r, K, RP, (__nv_bfloat16*)At);
}

// ===========================================================================
// The adapter's term of dX under dropout:  dX += D c (sU At^T), in place, bf16.
// A warp takes 16 tokens x 32 columns: the rank-r product on mma.m16n8k16 from
// 16-byte words of both factors (a lane's words hold the same eight j), through
// shared memory to eight consecutive columns a lane, one Philox block's mask.
// Bytes: dX read and written; the generator costs about as much (1111 x 3584: 14
// us).  sU may still be written when this grid starts, so plain loads read it after
// the wait; At is complete before the chain's first dependent launch.  dX is rounded
// to bf16 twice, here and by the product before: kept in fp32 between the two it
// would be twice the bytes.
// ===========================================================================
__global__ void __launch_bounds__(256, 3)
k_mx_rank_add(const __nv_bfloat16* sU, const __nv_bfloat16* __restrict__ At, int RP, int M, int K,
              __nv_bfloat16* dX, const __grid_constant__ DropoutKeys keys) {
  __shared__ __align__(16) float s_ad[8][16][36];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int m0 = (int)(blockIdx.x / (unsigned)(K / 32)) * 128 + warp * 16, k0 = (int)(blockIdx.x % (unsigned)(K / 32)) * 32;
  grid_launch_dependents();
  if (m0 >= M) return;
  grid_dependency_wait();
  float acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
  for (int j = 8 * t; j < RP; j += 32) {
    uint4 a[2], b[4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      a[h] = m0 + 8 * h + g < M ? *reinterpret_cast<const uint4*>(sU + (int64_t)(m0 + 8 * h + g) * RP + j)
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)                    // K % 32 == 0
      b[i] = __ldg(reinterpret_cast<const uint4*>(At + (int64_t)(k0 + 8 * i + g) * RP + j));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mma_16816(acc[i], a[0].x, a[1].x, a[0].y, a[1].y, b[i].x, b[i].y);
      mma_16816(acc[i], a[0].z, a[1].z, a[0].w, a[1].w, b[i].z, b[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2*>(&s_ad[warp][g + 8 * h][8 * i + 2 * t]) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = 8 * q + (lane >> 2), col = 8 * (lane & 3);
    if (m0 + row >= M) continue;
    const int64_t e = (int64_t)(m0 + row) * K + k0 + col;
    uint4 v = *reinterpret_cast<const uint4*>(dX + e);
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    const Draw draw = draw8((uint64_t)e >> 3, keys);
    const float* ad = &s_ad[warp][row][col];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = draw.keep(2 * i, keys.thr8) ? __fmaf_rn(ad[2 * i], keys.scale, bf16_lo(w[i])) : bf16_lo(w[i]);
      const float b = draw.keep(2 * i + 1, keys.thr8) ? __fmaf_rn(ad[2 * i + 1], keys.scale, bf16_hi(w[i])) : bf16_hi(w[i]);
      w[i] = pack_bf16x2(a, b);
    }
    *reinterpret_cast<uint4*>(dX + e) = v;
  }
}

void launch_mx_rank_add(const void* sU, const void* At, int RP, int M, int K, void* dX, const Dropout& drop,
                        cudaStream_t s) {
  const unsigned grid = (unsigned)(K / 32) * (unsigned)((M + 127) / 128);
  launch_dependent(k_mx_rank_add, dim3(grid), dim3(256), true, s, (const __nv_bfloat16*)sU, (const __nv_bfloat16*)At, RP, M, K,
                   (__nv_bfloat16*)dX, make_keys(drop));
}

}  // namespace qnf4
