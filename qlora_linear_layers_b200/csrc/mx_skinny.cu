// The adapter's products of the microscaled layer on the tensor cores:
//
//   down   S[M, r]  = Z[M, L] R[r, L]^T        T = X' A^T, and U = dY B from B^T
//   outer  G[C, r]  = Q[M, C]^T P[M, r]        dA^T from X' and s U, dB from dY and T
//
// Each reads a large bf16 matrix once and is bound by that read (r <= 128).  A
// CTA sums a tile of 128 rows (tokens, or columns of Q) x r in tensor memory,
// operands by TMA: for `down` both are K-major; for `outer` the contraction runs
// over the rows of both, so a tile of 64 tokens x 64 columns lands as an MN-major
// operand and the MMA transposes it (no transposed copy is made).  A cluster
// splits the contraction over 2^log_splits CTAs, so that few rows still occupy
// the GPU, and adds the partial sums through distributed shared memory in rank
// order: one launch, no workspace, the same bits every time.
//
//  * warp 0: TMA (a stage: 64 of the contraction, 16 KB + up to 16 KB);
//  * warp 1: tcgen05.mma kind::f16, M = 128, N = r (at least 16);
//  * warps 2-5: cluster reduction, rounding, stores.
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

namespace qnf4 {
namespace skinny {

using mx::elect_one;

constexpr int NS = 3;
constexpr int NUM_THREADS = 192;
constexpr int A_BYTES = 128 * 64 * 2, B_BYTES = 128 * 64 * 2;    // B at its largest

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
  int* status;
};

struct Smem {
  uint8_t a[NS][A_BYTES];   // a, then b: the partial sums of the reduction
  uint8_t b[NS][B_BYTES];
  uint64_t full[NS], empty[NS], acc_full;
  uint32_t tmem_base;
  int abort;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs an SM");
static_assert(128 * 128 * 4 <= NS * (A_BYTES + B_BYTES), "reduction buffer");

// MN-major operand with a 128-byte swizzle: 64 consecutive elements of a row are
// 128 bytes, eight rows 1024 bytes (the stride between groups of the
// contraction), the next 64 elements `group` bytes away.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t group) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(group >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

template <bool OUTER>
__global__ void __launch_bounds__(NUM_THREADS, 2)
k_mx_skinny(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_b0,
            const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b1,
            const __grid_constant__ Args g) {
  extern __shared__ uint8_t smem_raw[];
  Smem& S = *smem_align1024<Smem>(smem_raw);
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
    S.abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, 128);
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

  if (warp == 0) {
    if (elect_one()) {
      const int b_boxes = OUTER ? (g.N + 63) / 64 : 1;
      const uint32_t bytes = A_BYTES + (OUTER ? b_boxes * 8192 : g.N * 128);
      int s = 0, i = k0;
      uint32_t ph = 0;
      for (; i < k1; ++i) {
        if (!mbar_wait(&S.empty[s], ph ^ 1, abort, g.status)) break;
        mbar_arrive_expect_tx(&S.full[s], bytes);
        if (OUTER) {
          tma_load_2d(S.a[s], tm_a, &S.full[s], row0, i * 64);
          tma_load_2d(S.a[s] + 8192, tm_a, &S.full[s], row0 + 64, i * 64);
          for (int b = 0; b < b_boxes; ++b) tma_load_2d(S.b[s] + b * 8192, tm_b, &S.full[s], b * 64, i * 64);
        } else {
          tma_load_2d(S.a[s], tm_a, &S.full[s], i * 64, row0);
          tma_load_2d(S.b[s], tm_b, &S.full[s], i * 64, 0);
        }
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
                             (OUTER ? (1u << 15) | (1u << 16) : 0u);
      int s = 0;
      uint32_t ph = 0;
      for (int i = k0; i < k1; ++i) {
        if (!mbar_wait(&S.full[s], ph, abort, g.status)) break;
        tc_fence_after();
        const uint32_t aa = smem_u32(S.a[s]), bb = smem_u32(S.b[s]);
        const uint64_t a = OUTER ? mn_desc(aa, 8192) : sw128_kmajor_desc(aa);
        const uint64_t b = OUTER ? mn_desc(bb, 8192) : sw128_kmajor_desc(bb);
        constexpr uint32_t kStep = OUTER ? 2048 / 16 : 32 / 16;  // 16 rows, or 16 elements of a row
#pragma unroll
        for (int q = 0; q < 4; ++q) mma_ss(tmem, a + kStep * q, b + kStep * q, idesc, (i > k0 || q > 0) ? 1u : 0u);
        mma_commit(&S.empty[s]);
        if (++s == NS) { s = 0; ph ^= 1; }
      }
      mma_commit(&S.acc_full);
      mbar_wait(&S.acc_full, 0, abort, g.status);
    }
  } else {
    mbar_wait(&S.acc_full, 0, abort, g.status);
  }
  __syncwarp();
  cluster_sync();                                  // every rank is done with its stages
  const int quad = warp & 3;
  const int at = quad * 32 + lane, row = row0 + at;
  const int cs = g.N >> ls, lcs = __ffs(cs) - 1;   // columns each rank adds up (even)
  float* part = reinterpret_cast<float*>(S.a[0]);  // [splits][cs][128]
  if (warp >= 2) {
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < g.N; c += 16) {
      uint32_t v[16];
      tmem_ld16(tmem + ((uint32_t)(quad * 32) << 16) + c, v);
      tmem_wait_ld();
      const uint32_t mine = smem_u32(part + rank * cs * 128 + at);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        mx::st_cluster_f32(mapa_shared(mine + (uint32_t)(((c + j) & (cs - 1)) * 512), (c + j) >> lcs),
                           __uint_as_float(v[j]));
    }
  }
  cluster_sync();                                  // the partial sums have arrived
  if (warp >= 2 && row < p.rows) {
    const int col0 = rank * cs;
    const float f = OUTER ? p.s : 1.0f;
    const float div = !OUTER && p.row_scale ? p.row_scale[row] : 1.0f;
    for (int c = 0; c < cs; c += 2) {
      float v[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float* b = part + (c + j) * 128 + at;
        v[j] = b[0];
        for (int z = 1; z < splits; ++z) v[j] = __fadd_rn(v[j], b[z * cs * 128]);
      }
      const int col = col0 + c;
      if (OUTER) {
        if (col >= g.r) break;
        if (p.transposed) {
          p.out[(int64_t)col * p.rows + row] = __float2bfloat16_rn(__fmul_rn(f, v[0]));
          p.out[(int64_t)(col + 1) * p.rows + row] = __float2bfloat16_rn(__fmul_rn(f, v[1]));
        } else {
          *reinterpret_cast<uint32_t*>(p.out + (int64_t)row * g.r + col) =
              pack_bf16x2(__fmul_rn(f, v[0]), __fmul_rn(f, v[1]));
        }
      } else {
        float a = __fmul_rn(p.s, v[0]), b = __fmul_rn(p.s, v[1]);
        if (p.row_scale) { a = __fdiv_rn(a, div); b = __fdiv_rn(b, div); }
        if (p.pad) *reinterpret_cast<uint32_t*>(p.pad + (int64_t)row * g.RP + col) = pack_bf16x2(a, b);
        if (p.out && col < g.r) *reinterpret_cast<uint32_t*>(p.out + (int64_t)row * g.r + col) = pack_bf16x2(v[0], v[1]);
      }
    }
    if (!OUTER && p.pad && rank == 0)
      for (int c = g.N; c < g.RP; c += 8) *reinterpret_cast<uint4*>(p.pad + (int64_t)row * g.RP + c) = make_uint4(0, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

// Ranks of a cluster: up to about two CTAs an SM, at least four stages each.
static int log_splits_of(int tiles, int L, int num_sms) {
  const int nk = (L + 63) / 64;
  int ls = 0;
  while (ls < 3 && (tiles << (ls + 1)) <= 2 * num_sms && (nk >> (ls + 1)) >= 4) ++ls;
  return ls;
}

template <bool OUTER>
static int launch(const CUtensorMap& a0, const CUtensorMap& b0, const CUtensorMap& a1, const CUtensorMap& b1,
                  const Args& g, cudaStream_t s) {
  static std::atomic<unsigned long long> attr_devs{0};
  set_smem_attr_once(k_mx_skinny<OUTER>, (int)kSmemBytes, attr_devs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(g.p[0].tiles + g.p[1].tiles) << g.log_splits, 1, 1);
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1u << g.log_splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_mx_skinny<OUTER>, a0, b0, a1, b1, g) == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

}  // namespace skinny

int launch_mx_down(const void* Z, const void* R, int M, int L, int r, int RP, float s, const float* row_scale,
                   void* pad, void* out, int* status, cudaStream_t st, int num_sms) {
  using namespace skinny;
  Args g{};
  g.L = L;
  g.r = r;
  g.N = std::max(r, 16);
  g.RP = RP;
  g.status = status;
  g.p[0] = Problem{M, (M + 127) / 128, row_scale, (__nv_bfloat16*)pad, (__nv_bfloat16*)out, 0, s};
  g.log_splits = log_splits_of(g.p[0].tiles, L, num_sms);
  CUtensorMap a, b;
  if (!make_tmap_2d_bf16(&a, Z, L, M, L, 64, 128) || !make_tmap_2d_bf16(&b, R, L, r, L, 64, g.N)) return QLORA_ERR_CUDA;
  return launch<false>(a, b, a, b, g, st);
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
  g.log_splits = log_splits_of(g.p[0].tiles + g.p[1].tiles, M, num_sms);
  CUtensorMap a0, b0, a1, b1;
  if (!make_tmap_2d_bf16(&a0, Xd, K, M, K, 64, 64) || !make_tmap_2d_bf16(&b0, sU, r, M, ldu, 64, 64) ||
      !make_tmap_2d_bf16(&a1, dY, N, M, N, 64, 64) || !make_tmap_2d_bf16(&b1, T, r, M, r, 64, 64))
    return QLORA_ERR_CUDA;
  return launch<true>(a0, b0, a1, b1, g, st);
}

// ===========================================================================
// The backward's transposed adapter factors, in one launch:
//   At[K, RP] = A[r, K]^T, zero beyond r     Bt[r, N] = B[N, r]^T
// Tiles of 64 x r through shared memory (a row of 64 or r elements at a time).
// ===========================================================================
__global__ void __launch_bounds__(256)
k_mx_transpose(const __nv_bfloat16* __restrict__ A, const __nv_bfloat16* __restrict__ B, int r, int K, int N, int RP,
               __nv_bfloat16* __restrict__ At, __nv_bfloat16* __restrict__ Bt) {
  __shared__ __nv_bfloat16 tile[64][130];
  const int ka = (K + 63) / 64;
  const int tid = threadIdx.x;
  if ((int)blockIdx.x < ka) {
    const int k0 = blockIdx.x * 64;
    for (int i = tid; i < r * 64; i += 256) {
      const int j = i >> 6, k = i & 63;
      tile[k][j] = k0 + k < K ? A[(int64_t)j * K + k0 + k] : __nv_bfloat16();
    }
    __syncthreads();
    for (int i = tid; i < 64 * RP; i += 256) {
      const int k = i / RP, j = i % RP;
      if (k0 + k < K) At[(int64_t)(k0 + k) * RP + j] = j < r ? tile[k][j] : __float2bfloat16_rn(0.0f);
    }
  } else {
    const int n0 = ((int)blockIdx.x - ka) * 64;
    for (int i = tid; i < r * 64; i += 256) {
      const int n = i / r, j = i % r;
      tile[n][j] = n0 + n < N ? B[(int64_t)(n0 + n) * r + j] : __nv_bfloat16();
    }
    __syncthreads();
    for (int i = tid; i < r * 64; i += 256) {
      const int j = i >> 6, n = i & 63;
      if (n0 + n < N) Bt[(int64_t)j * N + n0 + n] = tile[n][j];
    }
  }
}

void launch_mx_transpose(const void* A, const void* B, int r, int K, int N, int RP, void* At, void* Bt,
                         cudaStream_t s) {
  k_mx_transpose<<<(K + 63) / 64 + (N + 63) / 64, 256, 0, s>>>((const __nv_bfloat16*)A, (const __nv_bfloat16*)B, r, K, N,
                                                               RP, (__nv_bfloat16*)At, (__nv_bfloat16*)Bt);
}

}  // namespace qnf4
