// Product of two microscaled 4-bit matrices on the block-scaled tensor cores:
//
//   Y[m, n] = rx[m] rw[n] * sum_b Sx[m, b] Sw[n, b] sum_{k in b} x[m, k] w[n, k]  (+ adapter)
//
// (NVFP4; MXFP4 has no row scales.)  The tensor core multiplies the E2M1
// elements and both block scales itself (tcgen05.mma kind::mxf4nvf4 /
// kind::mxf4) and sums in fp32, so nothing is expanded: a stage of 256
// contraction elements is 128 bytes a row.  The product is formed as
// Y^T = w x^T: 128 weight rows are the MMA's M, BN tokens its N, so one kernel
// serves one token (BN = 16) and thousands (BN = 256).
//
//  * warp 0: TMA loads of both operands' codes (128-byte swizzle) and plain
//    bulk copies of their scale tiles, one mbarrier a stage;
//  * warp 1: one thread copies a stage's scale tiles into tensor memory
//    (tcgen05.cp 32x128b, replicated to the four lane groups) and issues four
//    K = 64 MMAs.  Scale columns alternate between two slots; a slot is
//    written again only after the MMAs that read it have completed;
//  * warps 2-5: epilogue, tensor memory -> registers -> bf16.
//
// The adapter s (X A^T) B^T runs first, as RP / 64 bf16 K steps (kind::f16)
// into the same fp32 accumulator; its MMAs complete before the first
// block-scaled one is issued, since the two kinds need not run in order.
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
namespace mx {

constexpr int NUM_THREADS = 192;

template <int FMT, int BN>
struct Shape {
  static constexpr int NT = FMT == QLORA_NVFP4 ? 4 : 2;          // scale tiles of 256 elements
  static constexpr int RB = (BN + 127) / 128;                     // 128-row scale blocks of the tokens
  static constexpr int W_BYTES = BW * BKB, X_BYTES = BN * BKB;
  static constexpr int SW_BYTES = NT * 512, SX_BYTES = RB * NT * 512;
  static constexpr int STAGE = W_BYTES + X_BYTES + SW_BYTES + SX_BYTES;
  static constexpr int NS = BN > 128 ? 4 : BN > 64 ? 5 : 6;
  static constexpr int D_COLS = BN < 32 ? 32 : BN;
  static constexpr int SF_COLS = 4 * NT * (1 + RB);               // one slot: the stage's scale columns
  static constexpr int NEED = D_COLS + 2 * SF_COLS;
  static constexpr int TMEM_COLS = NEED <= 64 ? 64 : NEED <= 128 ? 128 : NEED <= 256 ? 256 : 512;
};

template <int FMT, int BN>
struct Smem {
  using Sh = Shape<FMT, BN>;
  uint8_t w[Sh::NS][Sh::W_BYTES];
  uint8_t x[Sh::NS][Sh::X_BYTES];
  uint8_t sw[Sh::NS][Sh::SW_BYTES];
  uint8_t sx[Sh::NS][Sh::SX_BYTES];
  float rx[BN];
  uint64_t full[Sh::NS], empty[Sh::NS], acc_full, kind;
  uint32_t tmem_base;
  int abort;
};

template <int FMT, int BN>
constexpr size_t smem_bytes() { return sizeof(Smem<FMT, BN>) + 1024; }

template <int FMT, int BN>
__global__ void __launch_bounds__(NUM_THREADS, 1)
k_mx_gemm(const __grid_constant__ CUtensorMap tm_w,       // [N, K / 2] bytes
          const __grid_constant__ CUtensorMap tm_x,       // [M, K / 2] bytes
          const __grid_constant__ CUtensorMap tm_sw,      // scale tiles of w
          const __grid_constant__ CUtensorMap tm_sx,      // scale tiles of x
          const __grid_constant__ CUtensorMap tm_wad,     // [N, RP] bf16
          const __grid_constant__ CUtensorMap tm_xad,     // [M, RP] bf16
          const Args p) {
  using Sh = Shape<FMT, BN>;
  constexpr int NS = Sh::NS, NT = Sh::NT, RB = Sh::RB;
  constexpr bool NV = FMT == QLORA_NVFP4;
  extern __shared__ uint8_t smem_raw[];
  auto& S = *smem_align1024<Smem<FMT, BN>>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * BW, m0 = blockIdx.y * BN;
  const int nk = (p.K + 255) / 256;
  const int nsteps = p.na + nk;

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
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  volatile int* abort = &S.abort;

  if (warp == 0) {
    if (elect_one()) {
      int i = 0;
      for (; i < nsteps; ++i) {
        const int s = i % NS;
        if (!mbar_wait(&S.empty[s], ((i / NS) & 1) ^ 1, abort, p.status)) break;
        if (i < p.na) {
          mbar_arrive_expect_tx(&S.full[s], Sh::W_BYTES + Sh::X_BYTES);
          tma_load_2d(S.w[s], &tm_wad, &S.full[s], i * 64, n0);
          tma_load_2d(S.x[s], &tm_xad, &S.full[s], i * 64, m0);
        } else {
          const int ks = i - p.na;
          mbar_arrive_expect_tx(&S.full[s], Sh::STAGE);
          tma_load_2d(S.w[s], &tm_w, &S.full[s], ks * BKB, n0);
          tma_load_2d(S.x[s], &tm_x, &S.full[s], ks * BKB, m0);
          tma_load_3d(S.sw[s], &tm_sw, &S.full[s], 0, ks * NT, n0 / 128);
          tma_load_3d(S.sx[s], &tm_sx, &S.full[s], 0, ks * NT, m0 / 128);
        }
      }
      if (i < nsteps || *abort)                                   // a wait gave up: let the copies in flight land
        for (int j = max(0, i - NS); j < i; ++j) drain_wait(&S.full[j % NS], (j / NS) & 1, p.status);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      constexpr uint32_t kId16 = idesc_bf16_f32(BW, BN);
      const uint32_t sf0 = tmem + Sh::D_COLS;
      const uint32_t sub = (uint32_t)(m0 % 128) / 32;            // token tile's place in its scale block
      bool ok = true;
      for (int i = 0; i < nsteps && ok; ++i) {
        const int s = i % NS;
        ok = mbar_wait(&S.full[s], (i / NS) & 1, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = sw128_kmajor_desc(smem_u32(S.w[s])), b = sw128_kmajor_desc(smem_u32(S.x[s]));
        if (i < p.na) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss(tmem, a + 2 * kk, b + 2 * kk, kId16, (i > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&S.empty[s]);
          if (i == p.na - 1) {
            mma_commit(&S.kind);
            ok = mbar_wait(&S.kind, 0, abort, p.status);
            tc_fence_after();
          }
          continue;
        }
        const int ks = i - p.na;
        if (ks >= 2) {                                            // this slot's last readers are done
          const int j = i - 2;
          ok = mbar_wait(&S.empty[j % NS], (j / NS) & 1, abort, p.status);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t sfw = sf0 + (ks & 1) * Sh::SF_COLS, sfx = sfw + 4 * NT;
        const int nq = min(4, (p.K - ks * 256 + 63) / 64);        // K = 64 steps with elements
        const int nt = NV ? nq : (nq + 1) / 2;
        for (int t = 0; t < nt; ++t) {
          scale_copy(sfw + 4 * t, scale_desc(smem_u32(S.sw[s] + t * 512)));
#pragma unroll
          for (int r = 0; r < RB; ++r)                            // a tile's token blocks side by side
            scale_copy(sfx + 4 * (RB * t + r), scale_desc(smem_u32(S.sx[s] + (r * NT + t) * 512)));
        }
        for (int q = 0; q < nq; ++q) {
          const int t = NV ? q : q >> 1;
          const uint32_t sf = NV ? 0u : 2u * (q & 1);
          mma_mx<FMT>(tmem, a + 2 * q, b + 2 * q, idesc_mx<FMT>(BW, BN, sf), sfw + 4 * t, sfx + 4 * RB * t + sub,
                      (i > 0 || q > 0) ? 1u : 0u);
        }
        mma_commit(&S.empty[s]);
      }
      mma_commit(&S.acc_full);
      mbar_wait(&S.acc_full, 0, abort, p.status);                 // nothing in flight when the CTA ends
    }
  } else {
    const int quad = warp & 3;
    const int n = n0 + quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    float rw = 1.0f;
    if (NV) {
      if (n < p.N) rw = p.wr[n];
      for (int i = threadIdx.x - 64; i < BN; i += 128) S.rx[i] = m0 + i < p.M ? p.xr[m0 + i] : 0.0f;
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
    if (mbar_wait(&S.acc_full, 0, abort, p.status)) {
      __syncwarp();
      tc_fence_after();
      const bool odd = lane & 1;
      const bool pairs = (p.N & 1) == 0;                          // two adjacent outputs share a 32-bit word
#pragma unroll 1
      for (int c = 0; c < BN; c += 16) {
        if (m0 + c >= p.M) break;
        uint32_t v[16];
        tmem_ld16(tmem + lanes + c, v);
        tmem_wait_ld();
        if (NV) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = __float_as_uint(__fmul_rn(__uint_as_float(v[j]), __fmul_rn(S.rx[c + j], rw)));
        }
        store_columns<16>(p, v, m0 + c, n, n - (odd ? 1 : 0), odd, pairs);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, Sh::TMEM_COLS);
  }
}

template <int FMT, int BN>
static int launch(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const void* tokad, const void* wad,
                  int RP, const Args& a, cudaStream_t s) {
  CUtensorMap tw, tx, tsw, tsx, twa, txa;
  const uint64_t kb = (uint64_t)a.K / 2;
  if (!make_tmap_2d_u8(&tw, w->packed, kb, a.N, kb, BKB, BW, true)) return QLORA_ERR_CUDA;
  if (!make_tmap_2d_u8(&tx, x->packed, kb, a.M, kb, BKB, BN, true)) return QLORA_ERR_CUDA;
  using Sh = Shape<FMT, BN>;
  if (!make_scale_tmap(&tsw, w->scales, FMT, a.N, a.K, Sh::NT, 1) ||
      !make_scale_tmap(&tsx, x->scales, FMT, a.M, a.K, Sh::NT, Sh::RB))
    return QLORA_ERR_CUDA;
  twa = tw;
  txa = tx;
  if (RP) {
    if (!make_tmap_2d_bf16(&twa, wad, RP, a.N, RP, 64, BW)) return QLORA_ERR_CUDA;
    if (!make_tmap_2d_bf16(&txa, tokad, RP, a.M, RP, 64, BN)) return QLORA_ERR_CUDA;
  }
  static std::atomic<unsigned long long> attr_devs{0};
  constexpr size_t bytes = smem_bytes<FMT, BN>();
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
  set_smem_attr_once(k_mx_gemm<FMT, BN>, (int)bytes, attr_devs);
  const dim3 grid((a.N + BW - 1) / BW, (a.M + BN - 1) / BN);
  k_mx_gemm<FMT, BN><<<grid, NUM_THREADS, bytes, s>>>(tw, tx, tsw, tsx, twa, txa, a);
  return QLORA_OK;
}

template <int FMT>
static int launch_fmt(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const void* tokad, const void* wad,
                      int RP, const Args& a, cudaStream_t s) {
  if (a.M <= 16) return launch<FMT, 16>(x, w, tokad, wad, RP, a, s);
  if (a.M <= 32) return launch<FMT, 32>(x, w, tokad, wad, RP, a, s);
  if (a.M <= 64) return launch<FMT, 64>(x, w, tokad, wad, RP, a, s);
  return launch<FMT, 128>(x, w, tokad, wad, RP, a, s);
}

}  // namespace mx

int launch_mx_gemm(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const void* tokad,
                   const void* wad, int RP, void* Y, int* status, cudaStream_t s, int num_sms) {
  mx::Args a{};
  a.xr = x->row_scale; a.wr = w->row_scale;
  a.out = static_cast<__nv_bfloat16*>(Y);
  a.M = (int)x->rows; a.N = (int)w->rows; a.K = (int)x->cols;
  a.na = RP / 64;
  a.status = status;
  if (a.M > 128) return mx::launch_gemm_pair(x, w, tokad, wad, RP, a, s, num_sms);
  return x->format == QLORA_NVFP4 ? mx::launch_fmt<QLORA_NVFP4>(x, w, tokad, wad, RP, a, s)
                                  : mx::launch_fmt<QLORA_MXFP4>(x, w, tokad, wad, RP, a, s);
}

}  // namespace qnf4
