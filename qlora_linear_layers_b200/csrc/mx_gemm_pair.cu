// Large products of two microscaled 4-bit matrices: pairs of SMs
// (tcgen05 cta_group::2), persistent.
//
//   Y^T tile = 256 weight rows x PN tokens; CTA r of a pair owns weight rows
//   128 r .. 128 r + 127 of the tile in its tensor memory and loads those rows
//   and PN / 2 of the tokens, so a stage (256 elements of K) brings half the
//   token codes to each SM.
//
// The tensor core is the bound.  In this kernel, and in a loop of its MMAs on two
// stages alone, one MMA (256 x PN x 64) takes 45 + PN / 2 cycles.  The pipe needs
// PN / 2 of them, and the bf16 kernel of gemm_pair.cu spends 137 on a tile of 224
// tokens, ramps included, so the 45 are not the hardware's least; what they go to is
// not known.  They make a tile as wide as the rounds of tiles allow (up to 256
// tokens), and the issuing thread has to keep up:
//  * a stage's 3 NT scale copies and 4 MMAs leave one thread in about 570
//    cycles (NVFP4) against 694 of MMA time; nothing else is in its loop;
//  * each pipeline stage has scale columns of its own in tensor memory (PN <=
//    256 accumulator columns leave 256, five stages of 48), so the "full"
//    barrier, which implies that the stage's last readers are done, is the only
//    wait of a stage;
//  * one accumulator: eight epilogue warps take it to registers as it is (128
//    values a thread), hand it back, and scale, round and store under the next
//    tile's MMAs.  They read it in the fragments that stmatrix transposes, so a
//    token's 32 outputs leave shared memory by TMA; stored from registers, a
//    4-byte word a lane, a tile's epilogue was longer than its MMAs (8192 x 18944
//    x 3584 NVFP4: 220 us against 181 us without stores).  Two accumulators would
//    hide that read too, but with tiles of 192 tokens, whose MMAs do 8 % less per
//    cycle.
// 8192 x 18944 x 3584 with r = 64: 211 us MXFP4, 219 us NVFP4 (5.4 and 5.2 PFLOP/s),
// 97 % of those cycles at the 1.64 GHz that the tensor cores' power leaves; the
// tensor pipe is active in 75 % of them.
// The adapter's bf16 K steps (kind::f16) come first and are complete before the
// block-scaled MMAs of the tile begin: MMAs of two kinds need not run in order.
// With one round of tiles the epilogue adds the adapter instead, on warp-level
// MMAs whose accumulator fragments are the ones it holds, while the tile's MMAs run
// (the layer of 512 x 4096 x 4096, r = 64: 15.3 us; 17.4 us after them).
//
// Every scale tile comes with the stage: each CTA loads the scales of its own
// 128 weight rows and of all PN tokens (one or two 128-row blocks), and the
// even CTA's tcgen05.cp moves both CTAs' copies to their tensor memories.
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

namespace qnf4 {
namespace mx {

constexpr int P_EPI = 8;                           // epilogue warps
constexpr int P_THREADS = 64 + 32 * P_EPI;         // warp 0 TMA, 1 MMA, 2-9 epilogue
constexpr uint16_t kBoth = 0x3;
template <int FMT, int PN>
struct PairShape {
  static_assert(PN % 64 == 0 && PN <= 256, "token tile");
  static constexpr int PNH = PN / 2;                              // tokens each CTA loads
  static constexpr int NT = FMT == QLORA_NVFP4 ? 4 : 2;           // scale tiles of 256 elements
  static constexpr int RB = PN == 128 ? 1 : 2;                    // 128-row scale blocks of the tokens
  static constexpr int W_BYTES = BW * BKB, X_BYTES = PNH * BKB;
  static constexpr int SW_BYTES = NT * 512, SX_BYTES = RB * NT * 512;
  static constexpr int NS = 5;
  static constexpr int SF_COLS = 4 * NT * (1 + RB);               // a stage's scale columns
  static_assert(PN + NS * SF_COLS <= 512, "tensor memory columns");
};

template <int FMT, int PN>
struct PairSmem {
  using Sh = PairShape<FMT, PN>;
  uint8_t w[Sh::NS][Sh::W_BYTES];
  uint8_t x[Sh::NS][Sh::X_BYTES];
  uint8_t sw[Sh::NS][Sh::SW_BYTES];
  uint8_t sx[Sh::NS][Sh::SX_BYTES];
  uint8_t out[P_EPI][2][kChunk * 64];              // a warp's chunks of kChunk tokens x 32 outputs
  float rx[2][PN];
  uint64_t full[Sh::NS], empty[Sh::NS], acc_full, acc_empty, kind, done;
  uint32_t tmem_base;
  int abort;
};

// A lane's values of a chunk times the row scales as they are stored: tokens m + 8 j +
// q, outputs n + 8 i.  Called for tiles with a scale far from 1; inline it takes
// registers from the tiles without.
static __device__ __noinline__ void times_far_scales_call(float* f, const float* xr, const float* wr, int m, int M, int n,
                                                          int N) {
  for (int e = 0; e < 32; ++e) {
    const int i = 2 * (e >> 4) + ((e >> 1) & 1), j = (e >> 2) & 3, q = e & 1;
    if (m + 8 * j + q < M && n + 8 * i < N) f[e] = times_scales(f[e], xr[m + 8 * j + q], wr[n + 8 * i], true);
  }
}
__device__ __forceinline__ void times_far_scales(float (&f)[2][4][4], const Args& p, int m, int n) {
  float t[32];                                     // a copy in memory, so that f stays in registers
#pragma unroll
  for (int e = 0; e < 32; ++e) t[e] = f[e >> 4][(e >> 2) & 3][e & 3];
  times_far_scales_call(t, p.xr, p.wr, m, p.M, n, p.N);
#pragma unroll
  for (int e = 0; e < 32; ++e) f[e >> 4][(e >> 2) & 3][e & 3] = t[e];
}

// ADD: the epilogue adds the adapter (p.r > 0).
template <int FMT, int PN, bool ADD>
__global__ void __launch_bounds__(P_THREADS, 1)
k_mx_gemm_pair(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
               const __grid_constant__ CUtensorMap tm_sw, const __grid_constant__ CUtensorMap tm_sx,
               const __grid_constant__ CUtensorMap tm_wad, const __grid_constant__ CUtensorMap tm_xad,
               const __grid_constant__ CUtensorMap tm_out, const Args p) {
  using Sh = PairShape<FMT, PN>;
  constexpr int NS = Sh::NS, NT = Sh::NT, RB = Sh::RB, PNH = Sh::PNH;
  constexpr bool NV = FMT == QLORA_NVFP4;
  extern __shared__ uint8_t smem_raw[];
  PairSmem<FMT, PN>& S =
      *reinterpret_cast<PairSmem<FMT, PN>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int tiles_n = (p.N + 2 * BW - 1) / (2 * BW);
  const int n_tiles = tiles_n * ((p.M + PN - 1) / PN);
  const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  const int nk = (p.K + 255) / 256;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&S.full[i], 1);                    // leader's expect_tx; bytes of both CTAs
      mbar_init(&S.empty[i], 1);                   // multicast commit
    }
    mbar_init(&S.acc_full, 1);                     // multicast commit
    mbar_init(&S.acc_empty, 2 * P_EPI);            // epilogue warps of both CTAs
    mbar_init(&S.kind, 1);
    mbar_init(&S.done, 1);
    S.abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&S.tmem_base, 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_sw);
    tma_prefetch_desc(&tm_sx);
  }
  tc_fence_before();
  cluster_sync();                                  // barriers of both CTAs initialised
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  volatile int* abort = &S.abort;

  if (warp == 0) {
    if (elect_one()) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      grid_dependency_wait();
      for (int tile = cluster; tile < n_tiles && ok; tile += n_clusters) {
        const int n0 = (tile % tiles_n) * (2 * BW) + (int)rank * BW;
        const int mt = (tile / tiles_n) * PN, m0 = mt + (int)rank * PNH;
        for (int i = -p.na; i < nk; ++i) {
          if (!(ok = mbar_wait_cluster(&S.empty[s], ph ^ 1, abort, p.status))) break;
          const uint32_t full0 = mapa_shared(smem_u32(&S.full[s]), 0);
          if (i < 0) {
            const int c = (i + p.na) * 64;
            if (leader) mbar_arrive_expect_tx(&S.full[s], 2 * (Sh::W_BYTES + Sh::X_BYTES));
            tma_load_2d_pair(S.w[s], &tm_wad, full0, c, n0);
            tma_load_2d_pair(S.x[s], &tm_xad, full0, c, m0);
          } else {
            if (leader)
              mbar_arrive_expect_tx(&S.full[s], 2 * (Sh::W_BYTES + Sh::X_BYTES + Sh::SW_BYTES + Sh::SX_BYTES));
            tma_load_2d_pair(S.w[s], &tm_w, full0, i * BKB, n0);
            tma_load_2d_pair(S.x[s], &tm_x, full0, i * BKB, m0);
            tma_load_3d_pair(S.sw[s], &tm_sw, full0, 0, i * NT, n0 / 128);
            tma_load_3d_pair(S.sx[s], &tm_sx, full0, 0, i * NT, mt / 128);
          }
          if (++s == NS) { s = 0; ph ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (leader && elect_one()) {
      constexpr uint32_t kId16 = idesc_bf16_f32(2 * BW, PN);
      const uint64_t a0 = sw128_kmajor_desc(smem_u32(S.w[0])), b0 = sw128_kmajor_desc(smem_u32(S.x[0]));
      const uint64_t sw0 = scale_desc(smem_u32(S.sw[0])), sx0 = scale_desc(smem_u32(S.sx[0]));
      int s = 0;
      uint32_t ph = 0, tp = 0;                     // stage, its phase; the tile's phase
      bool ok = true;
      grid_dependency_wait();                      // the bounded waits begin with the work
      for (int tile = cluster; tile < n_tiles && ok; tile += n_clusters, tp ^= 1) {
        // where the tokens' scales begin in their 128-row block's four columns: 0 or, with
        // tiles of 192, 2 (an odd one is a misaligned address)
        const uint32_t sub = (uint32_t)((tile / tiles_n) * PN % 128) / 32;
        ok = mbar_wait_cluster(&S.acc_empty, tp ^ 1, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        for (int i = 0; i < p.na; ++i) {
          if (!(ok = mbar_wait_cluster(&S.full[s], ph, abort, p.status))) break;
          tc_fence_after();
          const uint64_t a = a0 + (uint32_t)(s * (Sh::W_BYTES / 16)), b = b0 + (uint32_t)(s * (Sh::X_BYTES / 16));
#pragma unroll
          for (int q = 0; q < 4; ++q) mma_ss_pair(tmem, a + 2 * q, b + 2 * q, kId16, (i > 0 || q > 0) ? 1u : 0u);
          mma_commit_pair_mc(&S.empty[s], kBoth);
          if (++s == NS) { s = 0; ph ^= 1; }
        }
        if (ok && p.na > 0) {                      // the adapter's MMAs are complete
          mma_commit_pair_mc(&S.kind, 0x1);
          ok = mbar_wait_cluster(&S.kind, tp, abort, p.status);
          tc_fence_after();
        }
        if (!ok) break;
        for (int i = 0; i < nk; ++i) {
          if (!(ok = mbar_wait_cluster(&S.full[s], ph, abort, p.status))) break;
          tc_fence_after();
          const uint64_t a = a0 + (uint32_t)(s * (Sh::W_BYTES / 16)), b = b0 + (uint32_t)(s * (Sh::X_BYTES / 16));
          const uint64_t sw = sw0 + (uint32_t)(s * (Sh::SW_BYTES / 16)), sx = sx0 + (uint32_t)(s * (Sh::SX_BYTES / 16));
          const uint32_t sfw = tmem + PN + s * Sh::SF_COLS, sfx = sfw + 4 * NT;
          const int nq = min(4, (p.K - i * 256 + 63) / 64);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = NV ? q : q >> 1;         // scale tile of this K step
            if (q >= nq) break;
            if (NV || !(q & 1)) {
              scale_copy_pair(sfw + 4 * c, sw + 32 * c);
#pragma unroll
              for (int r = 0; r < RB; ++r) scale_copy_pair(sfx + 4 * (RB * c + r), sx + 32 * (r * NT + c));
            }
            mma_mx_pair<FMT>(tmem, a + 2 * q, b + 2 * q, idesc_mx<FMT>(2 * BW, PN, NV ? 0u : 2u * (q & 1)),
                             sfw + 4 * c, sfx + 4 * RB * c + sub, (i > 0 || q > 0 || p.na > 0) ? 1u : 0u);
          }
          mma_commit_pair_mc(&S.empty[s], kBoth);
          if (++s == NS) { s = 0; ph ^= 1; }
        }
        if (ok) mma_commit_pair_mc(&S.acc_full, kBoth);
      }
      mma_commit_pair_mc(&S.done, 0x1);            // every MMA has read its operands
      mbar_wait(&S.done, 0, abort, p.status);
    }
  } else {
    // warps (2 + e): lane quadrant warp % 4, column half e / 4
    constexpr int HC = PN / 2;
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + half * HC;
    const bool whole = (p.N & 7) == 0;             // rows of Y that TMA can store to
    const int e = warp - 2;
    const int g = lane >> 2;                       // fragment row
    const uint32_t acc_empty0 = mapa_shared(smem_u32(&S.acc_empty), 0);
    // this lane's row of the four blocks of a stmatrix: token lane % 8, outputs 8 (lane / 8) ..
    const uint32_t row_off = (uint32_t)((lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4));
    uint32_t tp = 0, buf = 0;
    bool ok = true;
    grid_dependency_wait();
    for (int tile = cluster; tile < n_tiles; tile += n_clusters, tp ^= 1) {
      const int nw = (tile % tiles_n) * (2 * BW) + (int)rank * BW + quad * 32;     // the warp's outputs
      const int mt = (tile / tiles_n) * PN, m0 = mt + half * HC;
      float rw[4] = {1.0f, 1.0f, 1.0f, 1.0f};
      bool far = false;
      if (NV) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (nw + 8 * i + g < p.N) rw[i] = p.wr[nw + 8 * i + g];
          far |= scale_far(rw[i]);
        }
        // the readers of this buffer, two tiles ago, passed the last tile's barrier
        for (int i = threadIdx.x - 64; i < PN; i += 32 * P_EPI) {
          const float rx = mt + i < p.M ? p.xr[mt + i] : 1.0f;
          S.rx[tp][i] = rx;
          far |= scale_far(rx);
        }
        // Scales far from 1 (times_scales) are applied by a pass of their own, and the
        // common one multiplies by 1: with both in it 4096^3 took 39.5 us, not 36.9.
        far = barrier_or<1, 32 * P_EPI>(far);
        if (far) {
#pragma unroll
          for (int i = 0; i < 4; ++i) rw[i] = 1.0f;
          for (int i = threadIdx.x - 64; i < PN; i += 32 * P_EPI) S.rx[tp][i] = 1.0f;
          asm volatile("bar.sync 1, %0;" :: "n"(32 * P_EPI) : "memory");
        }
      }
      // [chunk][16 outputs][8 tokens][fragment]: the accumulator, or the adapter's term
      constexpr int KEEP = ADD ? (HC / 32 < 3 ? HC / 32 : 3) : HC / 32;
      float v[KEEP][2][4][4];
      // the adapter's term of chunk c, B sT^T; a lane's words of both hold the same
      // eight k.  Up to three chunks are ready before the accumulator is (more spill).
      auto adapter = [&](float (&f)[2][4][4], int m) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) f[h][j][0] = f[h][j][1] = f[h][j][2] = f[h][j][3] = 0.0f;
        for (int k = 8 * (lane & 3); k - 8 * (lane & 3) < p.r; k += 32) {
          uint4 b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            b[i] = k < p.r && nw + 8 * i + g < p.N
                       ? __ldg(reinterpret_cast<const uint4*>(p.B + (int64_t)(nw + 8 * i + g) * p.r + k))
                       : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 t = k < p.r && m + 8 * j + g < p.M
                                ? *reinterpret_cast<const uint4*>(p.sT + (int64_t)(m + 8 * j + g) * p.r + k)
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mma_16816(f[h][j], b[2 * h].x, b[2 * h + 1].x, b[2 * h].y, b[2 * h + 1].y, t.x, t.y);
              mma_16816(f[h][j], b[2 * h].z, b[2 * h + 1].z, b[2 * h].w, b[2 * h + 1].w, t.z, t.w);
            }
          }
        }
      };
      if constexpr (ADD) {
#pragma unroll
        for (int c = 0; c < KEEP; ++c) adapter(v[c], m0 + 32 * c);
      }
      // after a wait that gave up the tiles pass without results, so that every
      // warp comes to every barrier
      if (!(ok = ok && mbar_wait_cluster(&S.acc_full, tp, abort, p.status))) continue;
      __syncwarp();
      tc_fence_after();
      if constexpr (!ADD) {
#pragma unroll
        for (int c = 0; c < HC / 32; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) tmem_ld_16x32(taddr + 32 * c + ((uint32_t)(16 * h) << 16), reinterpret_cast<uint32_t*>(v[c][h]));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty0);
        if (NV && far) {
#pragma unroll
          for (int c = 0; c < HC / 32; ++c) times_far_scales(v[c], p, m0 + 32 * c + 2 * (lane & 3), nw + g);
        }
      }
#pragma unroll
      for (int c = 0; c < HC / 32; ++c) {
        const int m = m0 + 32 * c;
        if (m >= p.M || nw >= p.N) break;
        float (&f)[2][4][4] = v[c < KEEP ? c : 0];
        [[maybe_unused]] float acc[2][4][4];       // ADD: one round, nobody waits for the accumulator
        if constexpr (ADD) {
          if (c >= KEEP) adapter(f, m);
#pragma unroll
          for (int h = 0; h < 2; ++h) tmem_ld_16x32(taddr + 32 * c + ((uint32_t)(16 * h) << 16), reinterpret_cast<uint32_t*>(acc[h]));
          tmem_wait_ld();
          if (NV && far) times_far_scales(acc, p, m + 2 * (lane & 3), nw + g);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 rx = make_float2(1.0f, 1.0f);
          if (NV) rx = *reinterpret_cast<const float2*>(&S.rx[tp][half * HC + 32 * c + 8 * j + 2 * (lane & 3)]);
#pragma unroll
          for (int i = 0; i < 4; ++i)              // outputs 8 i + g
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float& o = f[i >> 1][j][2 * (i & 1) + q];
              float x = ADD ? acc[i >> 1][j][2 * (i & 1) + q] : o;
              if (NV) x = __fmul_rn(x, __fmul_rn(q ? rx.y : rx.x, rw[i]));
              o = ADD ? __fadd_rn(x, o) : x;
            }
        }
        uint8_t* out = S.out[e][buf];
        buf ^= 1;                                  // across tiles too: one of 192 tokens has three chunks
        if (lane == 0) store_wait_read<1>();       // the store before the last one has left its chunk
        __syncwarp();
        const uint32_t to = smem_u32(out) + row_off;
#pragma unroll
        for (int j = 0; j < 4; ++j) {              // tokens 8 j .. 8 j + 7
          uint32_t o[4];                           // outputs 8 i .. 8 i + 7
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(f[i >> 1][j][2 * (i & 1)], f[i >> 1][j][2 * (i & 1) + 1]);
          stmatrix_x4_t(to + 512 * j, o[0], o[1], o[2], o[3]);
        }
        if (whole) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_out, out, nw, m);
            store_commit();
          }
        } else {
          // rows of Y without 16-byte boundaries: half a warp a token, 4-byte words where
          // they are aligned, so that a store of the warp touches two rows (2000 x 4097 x
          // 4096: 30 us, 90 us with a token a lane)
          __syncwarp();
          const int left = min(32, p.N - nw), l = lane & 15;
#pragma unroll 4
          for (int j = 0; j < 16; ++j) {
            const int t = 2 * j + (lane >> 4);
            const int64_t at = (int64_t)(m + t) * p.N + nw;
            const uint32_t w = *reinterpret_cast<const uint32_t*>(out + t * 64 + (((l >> 2) ^ ((t >> 1) & 3)) << 4) + (l & 3) * 4);
            const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w, 1);
            const int odd = (int)(at & 1), i = 2 * l + odd;
            const uint32_t v = odd ? prmt(w, next, 0x5432) : w;    // outputs i, i + 1
            if (m + t < p.M) {
              uint16_t* row = reinterpret_cast<uint16_t*>(p.out) + at;
              if (i + 1 < left) *reinterpret_cast<uint32_t*>(row + i) = v;
              else if (i < left) row[i] = (uint16_t)v;
              if (odd && l == 0) row[0] = (uint16_t)w;
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) store_wait_read<0>();           // the chunks outlive the stores that read them
  }

  if (warp == 0 && lane == 0 && *abort) {
    // a wait gave up: the copies in flight count on barriers that may never
    // complete, so give them a millisecond to land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  cluster_sync();                                  // both CTAs done with the paired TMEM
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Tokens of a tile: a round of tiles takes about nk stages of 4 (45 + PN / 2) measured
// cycles and 1000 for the accumulator's read and the ramp, so the cheapest of
// 128, 192 and 256 depends on how full it leaves the last round.
static int pair_tokens(const Args& a, int num_sms, int64_t* cycles) {
  const int pairs = std::max(1, num_sms / 2);
  int best = 256;
  *cycles = INT64_MAX;
  for (int pn : {256, 192, 128}) {
    const int64_t tiles = (int64_t)((a.N + 2 * BW - 1) / (2 * BW)) * ((a.M + pn - 1) / pn);
    const int64_t cost = (tiles + pairs - 1) / pairs * ((int64_t)(a.na + (a.K + 255) / 256) * 4 * (45 + pn / 2) + 1000);
    if (cost < *cycles) { *cycles = cost; best = pn; }
  }
  return best;
}

// Expected time in units of 10 ns: those cycles and 5.2 us of launch and ramp.
int64_t pair_cost(const Args& a, int num_sms) {
  int64_t cycles;
  pair_tokens(a, num_sms, &cycles);
  return 520 + cycles * 10 / 196;
}

int pair_rounds(const Args& a, int num_sms) {
  int64_t cycles;
  const int pn = pair_tokens(a, num_sms, &cycles);
  const int64_t tiles = (int64_t)((a.N + 2 * BW - 1) / (2 * BW)) * ((a.M + pn - 1) / pn);
  const int pairs = std::max(1, num_sms / 2);
  return (int)((tiles + pairs - 1) / pairs);
}

template <int FMT, int PN, bool ADD>
static int launch_pair(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const MxAdapter& ad, bool after_prep,
                       const Args& a, cudaStream_t s, int num_sms) {
  using Sh = PairShape<FMT, PN>;
  CUtensorMap tw, tx, tsw, tsx, twa, txa, to;
  const uint64_t kb = (uint64_t)a.K / 2;
  if (!make_tmap_2d_u8(&tw, w->packed, kb, a.N, kb, BKB, BW, true) ||
      !make_tmap_2d_u8(&tx, x->packed, kb, a.M, kb, BKB, Sh::PNH, true) ||
      !make_scale_tmap(&tsw, w->scales, FMT, a.N, a.K, Sh::NT, 1) ||
      !make_scale_tmap(&tsx, x->scales, FMT, a.M, a.K, Sh::NT, Sh::RB))
    return QLORA_ERR_CUDA;
  twa = tw;
  txa = tx;
  to = tw;
  if (a.N % 8 == 0 && !make_tmap_store_bf16(&to, a.out, a.N, a.M, kChunk)) return QLORA_ERR_CUDA;
  if (ad.RP && (!make_tmap_2d_bf16(&twa, ad.wt, ad.RP, a.N, ad.RP, 64, BW) ||
                !make_tmap_2d_bf16(&txa, ad.tok, ad.RP, a.M, ad.RP, 64, Sh::PNH)))
    return QLORA_ERR_CUDA;
  constexpr size_t bytes = sizeof(PairSmem<FMT, PN>) + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
  static std::atomic<unsigned long long> attr_devs{0};
  set_smem_attr_once(k_mx_gemm_pair<FMT, PN, ADD>, (int)bytes, attr_devs);
  const int tiles = ((a.N + 2 * BW - 1) / (2 * BW)) * ((a.M + PN - 1) / PN);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * std::max(1, std::min(tiles, num_sms / 2)), 1, 1);
  cfg.blockDim = dim3(P_THREADS, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after_prep ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_mx_gemm_pair<FMT, PN, ADD>, tw, tx, tsw, tsx, twa, txa, to, a) == cudaSuccess
             ? QLORA_OK : QLORA_ERR_CUDA;
}

template <int FMT>
static int launch_pair_fmt(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const MxAdapter& ad, bool after_prep,
                           const Args& a, cudaStream_t s, int num_sms) {
  int64_t cycles;
  const int pn = pair_tokens(a, num_sms, &cycles);
  if (a.r)
    return pn == 128   ? launch_pair<FMT, 128, true>(x, w, ad, after_prep, a, s, num_sms)
           : pn == 192 ? launch_pair<FMT, 192, true>(x, w, ad, after_prep, a, s, num_sms)
                       : launch_pair<FMT, 256, true>(x, w, ad, after_prep, a, s, num_sms);
  return pn == 128   ? launch_pair<FMT, 128, false>(x, w, ad, after_prep, a, s, num_sms)
         : pn == 192 ? launch_pair<FMT, 192, false>(x, w, ad, after_prep, a, s, num_sms)
                     : launch_pair<FMT, 256, false>(x, w, ad, after_prep, a, s, num_sms);
}

int launch_gemm_pair(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const MxAdapter& ad, bool after_prep,
                     const Args& a, cudaStream_t s, int num_sms) {
  return x->format == QLORA_NVFP4 ? launch_pair_fmt<QLORA_NVFP4>(x, w, ad, after_prep, a, s, num_sms)
                                  : launch_pair_fmt<QLORA_MXFP4>(x, w, ad, after_prep, a, s, num_sms);
}

}  // namespace mx
}  // namespace qnf4
