// Product of two microscaled 4-bit matrices on the block-scaled tensor cores:
//
//   Y[m, n] = rx[m] rw[n] * sum_b Sx[m, b] Sw[n, b] sum_{k in b} x[m, k] w[n, k]  (+ adapter)
//
// (NVFP4; MXFP4 has no row scales.)  The tensor core multiplies the E2M1
// elements and both block scales itself (tcgen05.mma kind::mxf4nvf4 /
// kind::mxf4) and sums in fp32, so nothing is expanded: a stage of 256
// contraction elements is 128 bytes a row.  The product is formed as
// Y^T = w x^T: weight rows are the MMA's M, tokens its N.
//
// This file: dispatch, and the kernel for few tokens, which reads the weight
// once and is bound by that read (or, below a few MB, by latency).  A tile is
// 128 weight rows x BN tokens (16, 32 or 128); a cluster of S CTAs splits its
// contraction, so that a few weight rows still occupy the GPU, and adds the
// partial sums through distributed shared memory in rank order: one launch, no
// workspace, the same bits every time.  Shared memory is sized for two CTAs an
// SM: one streams while the other one ramps or reduces.  One token, W 28672 x 8192
// MXFP4: 24.6 us, 5.1 TB/s.
//
//  * warp 0: TMA loads of both operands' codes (128-byte swizzle) and scale
//    tiles, one mbarrier a stage;
//  * warp 1: one thread copies a stage's scale tiles into the stage's own
//    tensor-memory columns (tcgen05.cp 32x128b, replicated to the four lane
//    groups) and issues four K = 64 MMAs;
//  * warps 2-5: epilogue, tensor memory -> cluster reduction -> bf16.
//
// The adapter's term s (X A^T) B^T comes from the epilogue warps, on warp-level
// MMAs while the others run (up to 32 tokens), or runs first, in rank 0, as RP /
// 64 bf16 K steps (kind::f16) into the same accumulator; these complete before the
// first block-scaled MMA is issued, since the two kinds need not run in order.
// Every wait is bounded (QLORA_ERR_TIMEOUT).

#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "gemm.h"
#include "mx.h"
#include "mx_mma.cuh"
#include "mx_gemm.cuh"

namespace qnf4 {
namespace mx {

constexpr int NUM_THREADS = 192;

template <int FMT, int BN>
struct Shape {
  static constexpr int NT = FMT == QLORA_NVFP4 ? 4 : 2;          // scale tiles of 256 elements
  static constexpr int W_BYTES = BW * BKB, X_BYTES = BN * BKB;
  static constexpr int S_BYTES = NT * 512;                        // scales of 128 rows
  static constexpr int STAGE = W_BYTES + X_BYTES + 2 * S_BYTES;
  static constexpr int NS = BN == 16 ? 4 : 3;                     // two CTAs an SM
  static constexpr bool OWN_PART = BN <= 32;                      // the partial sums have memory of their own
  static constexpr int ADD_PITCH = BW + 4;
  static constexpr int D_COLS = BN < 32 ? 32 : BN;
  static constexpr int SF_COLS = 8 * NT;                          // a stage's scale columns
  static constexpr int TMEM_COLS = 256;
  static_assert(D_COLS + NS * SF_COLS <= TMEM_COLS, "tensor memory columns");
};

template <int FMT, int BN>
struct Smem {
  using Sh = Shape<FMT, BN>;
  uint8_t w[Sh::NS][Sh::W_BYTES];                  // w, then x: the partial sums when !OWN_PART
  uint8_t x[Sh::NS][Sh::X_BYTES];
  uint8_t sw[Sh::NS][Sh::S_BYTES];
  uint8_t sx[Sh::NS][Sh::S_BYTES];
  float part[Sh::OWN_PART ? BN * 128 : 4];
  float add[Sh::OWN_PART ? BN * Sh::ADD_PITCH : 4];               // the adapter's term, [token][weight row]
  uint64_t full[Sh::NS], empty[Sh::NS], acc_full, kind;
  uint32_t tmem_base;
  int abort;
};

template <int FMT, int BN>
constexpr size_t smem_bytes() { return sizeof(Smem<FMT, BN>) + 1024; }

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The adapter's term of a warp's 32 weight rows, out[token][row] (pitch floats a
// token): B [32 rows, r] times sT [BN tokens, r], both bf16, on mma.m16n8k16.
// A lane takes 16-byte words of both operands, eight consecutive k each; the same
// k in both, so their order within the product does not matter.
template <int BN, int PITCH>
__device__ __forceinline__ void adapter_term(const __nv_bfloat16* B, int rows, const __nv_bfloat16* sT, int tokens,
                                             int r, float* out, int lane) {
  const int g = lane >> 2, t = lane & 3;
  float acc[2][BN / 8][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < BN / 8; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.0f;
  auto word = [&](const __nv_bfloat16* p, int row, int n, int k) {
    return row < n && k < r ? *reinterpret_cast<const uint4*>(p + (int64_t)row * r + k) : make_uint4(0, 0, 0, 0);
  };
  for (int k = 8 * t; k < r || k - 8 * t < r; k += 32) {
    uint4 a[2][2], x[BN / 8];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) a[i][h] = word(B, 16 * i + 8 * h + g, rows, k);
#pragma unroll
    for (int j = 0; j < BN / 8; ++j) x[j] = word(sT, 8 * j + g, tokens, k);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < BN / 8; ++j) {
        mma_16816(acc[i][j], a[i][0].x, a[i][1].x, a[i][0].y, a[i][1].y, x[j].x, x[j].y);
        mma_16816(acc[i][j], a[i][0].z, a[i][1].z, a[i][0].w, a[i][1].w, x[j].z, x[j].w);
      }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < BN / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)                  // row g or g + 8, token 2 t or 2 t + 1
        out[(8 * j + 2 * t + (e & 1)) * PITCH + 16 * i + g + 8 * (e >> 1)] = acc[i][j][e];
  __syncwarp();
}

template <int FMT, int BN>
__global__ void __launch_bounds__(NUM_THREADS, 2)
k_mx_gemm(const __grid_constant__ CUtensorMap tm_w,       // [N, K / 2] bytes
          const __grid_constant__ CUtensorMap tm_x,       // [M, K / 2] bytes
          const __grid_constant__ CUtensorMap tm_sw,      // scale tiles of w
          const __grid_constant__ CUtensorMap tm_sx,      // scale tiles of x
          const __grid_constant__ CUtensorMap tm_wad,     // [N, RP] bf16
          const __grid_constant__ CUtensorMap tm_xad,     // [M, RP] bf16
          const Args p, const int log_splits) {
  using Sh = Shape<FMT, BN>;
  constexpr int NS = Sh::NS, NT = Sh::NT;
  constexpr bool NV = FMT == QLORA_NVFP4;
  constexpr int kLogBN = BN == 16 ? 4 : BN == 32 ? 5 : 7;
  static_assert(BN * 512 <= NS * (Sh::W_BYTES + Sh::X_BYTES), "reduction buffer");
  extern __shared__ uint8_t smem_raw[];
  auto& S = *smem_align1024<Smem<FMT, BN>>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = 1 << log_splits;
  const int rank = (int)cluster_ctarank();
  const unsigned tile = blockIdx.x >> log_splits, tiles_n = (unsigned)(p.N + BW - 1) / BW;
  const int n0 = (int)(tile % tiles_n) * BW, m0 = (int)(tile / tiles_n) * BN;
  const int nk_all = (p.K + 255) / 256;
  const int k0 = (int)(((int64_t)nk_all * rank) >> log_splits), k1 = (int)(((int64_t)nk_all * (rank + 1)) >> log_splits);
  const int na = !Sh::OWN_PART && rank == 0 ? p.na : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    mbar_init(&S.acc_full, 1);
    mbar_init(&S.kind, 1);
    S.abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(&S.tmem_base, Sh::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_sw);
    tma_prefetch_desc(&tm_sx);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (splits > 1) cluster_arrive();                // a rank writes to another one once that one runs
  const uint32_t tmem = S.tmem_base;
  volatile int* abort = &S.abort;

  const int quad = warp & 3;
  const int n = n0 + quad * 32 + lane;             // an epilogue lane's weight row
  const int cs = BN >> log_splits;                 // token columns each rank adds up and stores (even)
  const int live = min(BN, p.M - m0);              // token columns that exist
  float rw = 1.0f;
  bool far = false;                                // a scale of the warp's rows and the tokens is (times_scales)
  if (warp == 0) {
    if (elect_one()) {
      int s = 0, i = -na;
      uint32_t ph = 0;
      // the first stages' weight loads do not wait for the grid that writes x
      const int ahead = na ? 0 : min(NS, k1 - k0);
      for (int j = 0; j < ahead; ++j) {
        mbar_arrive_expect_tx(&S.full[j], Sh::STAGE);
        tma_load_2d(S.w[j], &tm_w, &S.full[j], (k0 + j) * BKB, n0);
        tma_load_3d(S.sw[j], &tm_sw, &S.full[j], 0, (k0 + j) * NT, n0 / 128);
      }
      grid_dependency_wait();
      for (; i < k1 - k0; ++i) {
        if (!mbar_wait(&S.empty[s], ph ^ 1, abort, p.status)) break;
        if (i < 0) {
          mbar_arrive_expect_tx(&S.full[s], Sh::W_BYTES + Sh::X_BYTES);
          tma_load_2d(S.w[s], &tm_wad, &S.full[s], (i + na) * 64, n0);
          tma_load_2d(S.x[s], &tm_xad, &S.full[s], (i + na) * 64, m0);
        } else {
          const int ks = k0 + i;
          if (i >= ahead) {
            mbar_arrive_expect_tx(&S.full[s], Sh::STAGE);
            tma_load_2d(S.w[s], &tm_w, &S.full[s], ks * BKB, n0);
            tma_load_3d(S.sw[s], &tm_sw, &S.full[s], 0, ks * NT, n0 / 128);
          }
          tma_load_2d(S.x[s], &tm_x, &S.full[s], ks * BKB, m0);
          tma_load_3d(S.sx[s], &tm_sx, &S.full[s], 0, ks * NT, m0 / 128);
        }
        if (++s == NS) { s = 0; ph ^= 1; }
      }
      if (*abort) {                                               // a wait gave up: let the copies in flight land
        const int n = na + i;
        for (int j = max(0, n - NS); j < n; ++j) drain_wait(&S.full[j % NS], (j / NS) & 1, p.status);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      constexpr uint32_t kId16 = idesc_bf16_f32(BW, BN);
      const uint64_t a0 = sw128_kmajor_desc(smem_u32(S.w[0])), b0 = sw128_kmajor_desc(smem_u32(S.x[0]));
      const uint64_t sw0 = scale_desc(smem_u32(S.sw[0])), sx0 = scale_desc(smem_u32(S.sx[0]));
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      grid_dependency_wait();                      // the bounded waits begin with the work
      for (int i = -na; i < k1 - k0; ++i) {
        ok = mbar_wait(&S.full[s], ph, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = a0 + (uint32_t)(s * (Sh::W_BYTES / 16)), b = b0 + (uint32_t)(s * (Sh::X_BYTES / 16));
        if (i < 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q) mma_ss(tmem, a + 2 * q, b + 2 * q, kId16, (i > -na || q > 0) ? 1u : 0u);
          mma_commit(&S.empty[s]);
          if (i == -1) {
            mma_commit(&S.kind);
            ok = mbar_wait(&S.kind, 0, abort, p.status);
            if (!ok) break;
            tc_fence_after();
          }
        } else {
          const uint64_t sw = sw0 + (uint32_t)(s * (Sh::S_BYTES / 16)), sx = sx0 + (uint32_t)(s * (Sh::S_BYTES / 16));
          const uint32_t sfw = tmem + Sh::D_COLS + s * Sh::SF_COLS, sfx = sfw + 4 * NT;
          const int nq = min(4, (p.K - (k0 + i) * 256 + 63) / 64);  // K = 64 steps with elements
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = NV ? q : q >> 1;                        // scale tile of this K step
            if (q >= nq) break;
            if (NV || !(q & 1)) {
              scale_copy(sfw + 4 * c, sw + 32 * c);
              scale_copy(sfx + 4 * c, sx + 32 * c);
            }
            mma_mx<FMT>(tmem, a + 2 * q, b + 2 * q, idesc_mx<FMT>(BW, BN, NV ? 0u : 2u * (q & 1)), sfw + 4 * c,
                        sfx + 4 * c, (i > 0 || q > 0 || na > 0) ? 1u : 0u);
          }
          mma_commit(&S.empty[s]);
        }
        if (++s == NS) { s = 0; ph ^= 1; }
      }
      mma_commit(&S.acc_full);
      mbar_wait(&S.acc_full, 0, abort, p.status);                 // nothing in flight when the CTA ends
    }
  } else {
    grid_dependency_wait();
    if (NV) {
      if (n < p.N) rw = p.wr[n];
      far = scale_far(rw);
      for (int c = lane; c < live; c += 32) far |= scale_far(p.xr[m0 + c]);
      far = __any_sync(0xFFFFFFFFu, far);
    }
    if constexpr (Sh::OWN_PART) {                  // the adapter, while the MMAs run
      const int row = n0 + quad * 32;
      if (p.r && row < p.N)
        adapter_term<BN, Sh::ADD_PITCH>(p.B + (int64_t)row * p.r, min(32, p.N - row), p.sT + (int64_t)m0 * p.r,
                                        p.M - m0, p.r, S.add + quad * 32, lane);
    }
    mbar_wait(&S.acc_full, 0, abort, p.status);
  }
  __syncwarp();
  if (splits > 1) {
    cluster_wait();
    if (!Sh::OWN_PART) cluster_sync();             // every rank is done with its stages
  }
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;
  const bool odd = lane & 1;
  const bool pairs = (p.N & 1) == 0;
  float* part = Sh::OWN_PART ? S.part : reinterpret_cast<float*>(S.w[0]);   // [splits][cs][128]
  if (warp >= 2) {
    tc_fence_after();
    if (splits == 1) {
#pragma unroll 1
      for (int c = 0; c < live; c += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + lanes + c, v);
        tmem_wait_ld();
        if (NV) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float rx = c + j < live ? p.xr[m0 + c + j] : 0.0f;
            v[j] = __float_as_uint(times_scales(__uint_as_float(v[j]), rx, rw, far));
          }
        }
        if (Sh::OWN_PART && p.r) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = __float_as_uint(__fadd_rn(__uint_as_float(v[j]), S.add[(c + j) * Sh::ADD_PITCH + quad * 32 + lane]));
        }
        store_columns<16>(p, v, m0 + c, n, n - (odd ? 1 : 0), odd, pairs);
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < live; c += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + lanes + c, v);
        tmem_wait_ld();
        const uint32_t mine = smem_u32(part + rank * cs * 128 + quad * 32 + lane);
        const int lcs = kLogBN - log_splits;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < live)
            st_cluster_f32(mapa_shared(mine + (uint32_t)(((c + j) & (cs - 1)) * 512), (c + j) >> lcs),
                           __uint_as_float(v[j]));
      }
    }
  }
  if (splits > 1) {
    cluster_sync();                                // the partial sums have arrived
    if (warp >= 2) {
      const float* mine = part + quad * 32 + lane;
      const int first = m0 + rank * cs, n_cols = min(cs, p.M - first);
      const float* add = Sh::OWN_PART && p.r ? S.add + rank * cs * Sh::ADD_PITCH + quad * 32 + lane : nullptr;
      if (cs >= 8)
        for (int c = 0; c < n_cols; c += 8)
          add_ranks<8, NV>(p, mine + c * 128, cs * 128, splits, first + c, n, rw, far, add ? add + c * Sh::ADD_PITCH : nullptr,
                           Sh::ADD_PITCH, odd, pairs);
      else
        for (int c = 0; c < n_cols; c += 2)
          add_ranks<2, NV>(p, mine + c * 128, cs * 128, splits, first + c, n, rw, far, add ? add + c * Sh::ADD_PITCH : nullptr,
                           Sh::ADD_PITCH, odd, pairs);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::TMEM_COLS);
  }
}

// Expected time of this kernel in units of 10 ns, with 2^*log_splits ranks a
// tile (1 to 8, as many as keep at most about one CTA on each SM, when that is
// faster).  Fitted on B200 to W 4096 x 4096, 1024 x 18944 and 3584 x 18944 for
// 1 to 128 tokens: 3.3 us of launch, ramp and drain (4.6 with 128 tokens), 0.34
// us a stage (0.5), and 1.8 us + 30 ns a token for the cluster's reduction (4.2).
// E.g. W 4096 x 4096, one token: 8.9 us unsplit, 7.7, 6.9 and 7.4 with 2, 4 and
// 8 ranks; W 18944 x 3584 (148 tiles), 16 tokens: 10.4 us unsplit, 11.4 split.
static int64_t split_cost(const Args& a, int bn, int num_sms, int* log_splits) {
  const int64_t tiles = (int64_t)((a.N + BW - 1) / BW) * ((a.M + bn - 1) / bn);
  const int nk = (a.K + 255) / 256;
  int64_t best = INT64_MAX;
  for (int s = 0; s <= 3 && (nk >> s) > 0; ++s) {
    if (s && (tiles << s) > num_sms + num_sms / 8) break;
    const int64_t waves = s ? 1 : (tiles + num_sms - 1) / num_sms;
    const int64_t stages = a.na + (nk + (1 << s) - 1) / (1 << s);
    const int64_t cost = bn > 32 ? 460 + waves * stages * 50 + (s ? 420 : 0)
                                 : 330 + waves * stages * 34 + (s ? 180 + 3 * bn : 0);
    if (cost < best) { best = cost; *log_splits = s; }
  }
  return best;
}

template <int FMT, int BN>
static int launch(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const MxAdapter& ad, bool after_prep,
                  const Args& a, cudaStream_t s, int num_sms) {
  using Sh = Shape<FMT, BN>;
  CUtensorMap tw, tx, tsw, tsx, twa, txa;
  const uint64_t kb = (uint64_t)a.K / 2;
  if (!make_tmap_2d_u8(&tw, w->packed, kb, a.N, kb, BKB, BW, true) ||
      !make_tmap_2d_u8(&tx, x->packed, kb, a.M, kb, BKB, BN, true) ||
      !make_scale_tmap(&tsw, w->scales, FMT, a.N, a.K, Sh::NT, 1) ||
      !make_scale_tmap(&tsx, x->scales, FMT, a.M, a.K, Sh::NT, 1))
    return QLORA_ERR_CUDA;
  twa = tw;
  txa = tx;
  if (ad.RP && (!make_tmap_2d_bf16(&twa, ad.wt, ad.RP, a.N, ad.RP, 64, BW) ||
                !make_tmap_2d_bf16(&txa, ad.tok, ad.RP, a.M, ad.RP, 64, BN)))
    return QLORA_ERR_CUDA;
  constexpr size_t bytes = smem_bytes<FMT, BN>();
  static_assert(2 * (bytes + 1024) <= 228 * 1024, "two CTAs an SM");
  static std::atomic<unsigned long long> attr_devs{0};
  set_smem_attr_once(k_mx_gemm<FMT, BN>, (int)bytes, attr_devs);
  int log_splits = 0;
  split_cost(a, BN, num_sms, &log_splits);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + BW - 1) / BW) * (unsigned)((a.M + BN - 1) / BN) << log_splits, 1, 1);
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1u << log_splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after_prep ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_mx_gemm<FMT, BN>, tw, tx, tsw, tsx, twa, txa, a, log_splits) == cudaSuccess
             ? QLORA_OK : QLORA_ERR_CUDA;
}

template <int FMT>
static int launch_fmt(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const MxAdapter& ad, bool after_prep,
                      const Args& a, cudaStream_t s, int num_sms) {
  if (a.M <= 16) return launch<FMT, 16>(x, w, ad, after_prep, a, s, num_sms);
  if (a.M <= 32) return launch<FMT, 32>(x, w, ad, after_prep, a, s, num_sms);
  return launch<FMT, 128>(x, w, ad, after_prep, a, s, num_sms);
}

}  // namespace mx

bool mx_adapter_in_epilogue(int M, int N, int K, int num_sms) {
  mx::Args a{};
  a.M = M; a.N = N; a.K = K;
  int ls = 0;
  return M <= mx::kFewTokens ||
         (mx::pair_rounds(a, num_sms) == 1 && mx::pair_cost(a, num_sms) <= mx::split_cost(a, 128, num_sms, &ls));
}

int launch_mx_gemm(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const MxAdapter& ad, bool after_prep, void* Y,
                   int* status, cudaStream_t s, int num_sms) {
  mx::Args a{};
  a.xr = x->row_scale; a.wr = w->row_scale;
  a.out = static_cast<__nv_bfloat16*>(Y);
  a.M = (int)x->rows; a.N = (int)w->rows; a.K = (int)x->cols;
  a.na = ad.RP / 64;
  a.r = ad.r;
  a.sT = static_cast<const __nv_bfloat16*>(ad.sT);
  a.B = static_cast<const __nv_bfloat16*>(ad.B);
  a.status = status;
  // Up to 32 tokens the weight's read bounds the product.  From 33 the paired
  // kernel is faster wherever it has tiles enough (W 4096 x 4096, 128 tokens:
  // 9.2 us against 10.6), a split contraction where a long one meets few weight
  // rows (W 1024 x 18944, 128 tokens: 12.7 us against 23.1).
  int ls = 0;
  if (a.M > mx::kFewTokens && mx::pair_cost(a, num_sms) <= mx::split_cost(a, 128, num_sms, &ls))
    return mx::launch_gemm_pair(x, w, ad, after_prep, a, s, num_sms);
  return x->format == QLORA_NVFP4 ? mx::launch_fmt<QLORA_NVFP4>(x, w, ad, after_prep, a, s, num_sms)
                                  : mx::launch_fmt<QLORA_MXFP4>(x, w, ad, after_prep, a, s, num_sms);
}

}  // namespace qnf4
