// dX of the microscaled layer for few and middling token counts, the weight
// expanded inside the product:
//
//   dX^T[k, m] = sum_n W'[n, k] dY[m, n] (+ sum_j A[j, k] sU[m, j])
//
// The contraction runs over the weight's rows, so a tile of 64 rows x 128 columns
// is an MN-major operand as it lies: eight converter warps turn its codes into
// bf16 (the values of qlora_mx_dequantize, a row's block scale once for 16 or 32
// values) and store them with the 128-byte swizzle, nothing is transposed and no
// bf16 copy of the weight exists.  The adapter's A [r, K] is MN-major too and
// arrives by TMA, like dY and sU (K-major).
//
//  * warp 0: TMA; warp 1: tcgen05.mma kind::f16, M = 128 columns of W, N = BN
//    tokens; warps 2-5: epilogue; warps 6-21: converters, two groups of eight warps
//    on alternate stages, each thread one row's 32 codes, loaded kAhead of its
//    stages ahead (one group alone: 1000 cycles a stage, its chain of loads,
//    conversion and fence).
//  * a cluster splits the contraction over 2^log_splits CTAs and adds the partial
//    sums through distributed shared memory in rank order; or, unsplit, is a pair of
//    SMs (tcgen05 cta_group::2) with a tile of 256 columns x 256 tokens, each
//    expanding its own 128 columns and loading half of the tokens.
//
// Bound: a stage is 4 (45 + BN / 2) cycles of MMA (692 at 256 tokens; the pipe needs 4
// BN / 2 of them, see mx_gemm_pair.cu), about 400 of converter issue, and at 256
// tokens 96 KB of shared-memory traffic (750 cycles; 64 KB in a pair: W 18944 x 3584,
// 1111 tokens 140 us against 150, 470 ns a stage at the clock that the tensor cores'
// power leaves).  Every tile of tokens expands the weight again, so from some token
// count on the expansion to HBM and the paired-SM GEMM are cheaper (cost_expanded).
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
#include "mx_values.cuh"

namespace qnf4 {
namespace dx {

using namespace mx;

constexpr int kConv = 8;                           // converter warps of a group
constexpr int kGroups = 2;
constexpr int NUM_THREADS = 32 * (6 + kGroups * kConv);
constexpr int kAhead = 1;                          // of its stages that a converter's loads run ahead
constexpr int A_BYTES = 64 * 128 * 2;

struct DxArgs {
  Args out;                 // out [M, N = columns of W]
  const uint8_t* packed;
  const uint8_t* scales;
  const float* row_scale;
  int rows;                 // of W: the contraction
  int na;                   // adapter steps of 64
  int log_splits;
  int* status;
};

// PAIR: two CTAs on paired SMs share a tile of 256 columns x BN tokens, each with
// its 128 columns of W and half of the tokens.
template <int BN, bool PAIR>
struct Shape {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int B_ROWS = BN / kCtas;        // tokens of a CTA's loads
  static constexpr int B_BYTES = B_ROWS * 128;
  static constexpr int NS = B_ROWS > 128 ? 4 : 6;
  static constexpr int D_COLS = BN < 32 ? 32 : BN;
};

template <int BN, bool PAIR>
struct Smem {
  using Sh = Shape<BN, PAIR>;
  uint8_t a[Sh::NS][A_BYTES];                      // a, then b: the partial sums of the reduction
  uint8_t b[Sh::NS][Sh::B_BYTES];
  uint8_t out[4][2][kChunk * 64];                  // an epilogue warp's chunks
  uint64_t full_a[Sh::NS], full_b[Sh::NS], empty[Sh::NS], acc_full;
  uint32_t tmem_base;
  int abort;
};

template <int FMT, int BN, bool PAIR>
__global__ void __launch_bounds__(NUM_THREADS, 1)
k_mx_dx(const __grid_constant__ CUtensorMap tm_dy,         // [M, rows of W] bf16
        const __grid_constant__ CUtensorMap tm_a,          // [r, K] bf16
        const __grid_constant__ CUtensorMap tm_su,         // [M, RP] bf16
        const __grid_constant__ CUtensorMap tm_out,        // [M, K] bf16
        const DxArgs g) {
  using Sh = Shape<BN, PAIR>;
  constexpr int NS = Sh::NS, P = Sh::kCtas;
  static_assert(BN * 512 <= NS * (A_BYTES + Sh::B_BYTES), "reduction buffer");
  extern __shared__ uint8_t smem_raw[];
  grid_launch_dependents();
  Smem<BN, PAIR>& S = *smem_align1024<Smem<BN, PAIR>>(smem_raw);
  const Args& p = g.out;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ls = PAIR ? 0 : g.log_splits, splits = 1 << ls;
  const int half = PAIR ? (int)cluster_ctarank() : 0, rank = PAIR ? 0 : (int)cluster_ctarank();
  const bool leader = half == 0;
  const unsigned tile = blockIdx.x >> ls, tiles_c = (unsigned)((p.N + 128 * P - 1) / (128 * P) * P);
  const int c0 = (int)(tile % tiles_c) * 128;                                // columns of W
  const int m0 = (int)(tile / tiles_c) * BN, mb = m0 + half * Sh::B_ROWS;    // tokens
  const int nk_all = (g.rows + 63) / 64;
  const int k0 = (int)(((int64_t)nk_all * rank) >> ls), k1 = (int)(((int64_t)nk_all * (rank + 1)) >> ls);
  const int na = rank == 0 ? g.na : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&S.full_a[i], P * kConv);          // a pair's: the leader's, for both
      mbar_init(&S.full_b[i], 1);
      mbar_init(&S.empty[i], 1);
    }
    mbar_init(&S.acc_full, 1);
    S.abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(&S.tmem_base, Sh::D_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&S.tmem_base, Sh::D_COLS);
      tmem_relinquish();
    }
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_dy);
    tma_prefetch_desc(&tm_out);
  }
  tc_fence_before();
  if (PAIR) cluster_sync();                        // barriers of both CTAs initialised
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  volatile int* abort = &S.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return PAIR ? mbar_wait_cluster(bar, parity, abort, g.status) : mbar_wait(bar, parity, abort, g.status);
  };
  // where the wait may begin while the kernel before, which writes sU, still runs
  auto wait_after_grid = [&](uint64_t* bar, uint32_t parity) {
    return PAIR ? mbar_wait_cluster<true>(bar, parity, abort, g.status) : mbar_wait<true>(bar, parity, abort, g.status);
  };
  auto load_tile = [&](void* dst, const CUtensorMap* t, uint64_t* bar, int x, int y) {
    if (PAIR) tma_load_2d_pair(dst, t, mapa_shared(smem_u32(bar), 0), x, y);
    else tma_load_2d(dst, t, bar, x, y);
  };
  auto commit = [&](uint64_t* bar) {
    if (PAIR) mma_commit_pair_mc(bar, 0x3);
    else mma_commit(bar);
  };

  if (warp == 0) {
    if (elect_one()) {
      int s = 0, i = -na;
      uint32_t ph = 0;
      if (na) grid_dependency_wait();              // sU comes from the kernel before
      for (; i < k1 - k0; ++i) {
        if (!wait(&S.empty[s], ph ^ 1)) break;
        if (i < 0) {
          if (leader) mbar_arrive_expect_tx(&S.full_b[s], P * (A_BYTES + Sh::B_BYTES));
          load_tile(S.a[s], &tm_a, &S.full_b[s], c0, (i + na) * 64);
          load_tile(S.a[s] + 8192, &tm_a, &S.full_b[s], c0 + 64, (i + na) * 64);
          load_tile(S.b[s], &tm_su, &S.full_b[s], (i + na) * 64, mb);
        } else {
          if (leader) mbar_arrive_expect_tx(&S.full_b[s], P * Sh::B_BYTES);
          load_tile(S.b[s], &tm_dy, &S.full_b[s], (k0 + i) * 64, mb);
        }
        if (++s == NS) { s = 0; ph ^= 1; }
      }
      if (!PAIR && *abort) {                       // a wait gave up: let the copies in flight land
        const int n = na + i;
        for (int j = max(0, n - NS); j < n; ++j) drain_wait(&S.full_b[j % NS], (j / NS) & 1, g.status);
      }
    }
  } else if (warp == 1) {
    if (leader && elect_one()) {
      constexpr uint32_t idesc = idesc_bf16_f32(128 * P, BN) | (1u << 15);   // A is MN-major
      int s = 0;
      uint32_t ph = 0;
      for (int i = -na; i < k1 - k0; ++i) {
        if (!wait_after_grid(&S.full_b[s], ph)) break;
        // the converters never fill the first na slots' first use (na <= 2 < NS)
        if (i >= 0 && !wait(&S.full_a[s], ph ^ (s < na ? 1u : 0u))) break;
        tc_fence_after();
        const uint64_t a = mn_desc(smem_u32(S.a[s]), 8192), b = sw128_kmajor_desc(smem_u32(S.b[s]));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t add = (i > -na || q > 0) ? 1u : 0u;
          if (PAIR) mma_ss_pair(tmem, a + 128 * q, b + 2 * q, idesc, add);
          else mma_ss(tmem, a + 128 * q, b + 2 * q, idesc, add);
        }
        commit(&S.empty[s]);
        if (++s == NS) { s = 0; ph ^= 1; }
      }
      commit(&S.acc_full);
      wait(&S.acc_full, 0);
    }
  } else if (warp >= 6) {
    // thread (row, q): columns 32 q .. 32 q + 31 of the tile's row, one of a warp's 32
    // consecutive rows, so that eight lanes store to eight swizzled positions
    const int group = (warp - 6) / kConv;
    const int ct = threadIdx.x - 32 * (6 + group * kConv), row = ct & 63, q = ct >> 6;
    const int kc = c0 + 32 * q;
    const int64_t tiles = mx_scale_tiles(FMT, p.N);
    const int n_st = k1 - k0;
    uint4 cw[kAhead];
    uint32_t sc[kAhead];
    float rs[kAhead];
    auto load = [&](int i, int d) {
      const int n = (k0 + i) * 64 + row;
      cw[d] = make_uint4(0, 0, 0, 0);
      sc[d] = 0;
      rs[d] = 1.0f;
      if (i < n_st && n < g.rows && kc < p.N) {
        cw[d] = __ldg(reinterpret_cast<const uint4*>(g.packed + (int64_t)n * (p.N / 2) + kc / 2));
        if (FMT == QLORA_NVFP4) {
          sc[d] = __ldg(reinterpret_cast<const uint16_t*>(g.scales + mx_scale_offset(n, kc / 16, tiles)));
          rs[d] = __ldg(g.row_scale + n);
        } else {
          sc[d] = __ldg(g.scales + mx_scale_offset(n, kc / 32, tiles));
        }
      }
    };
#pragma unroll
    for (int d = 0; d < kAhead; ++d) load(group + kGroups * d, d);
    const uint32_t base = (uint32_t)((q >> 1) * 8192 + row * 128);
    int s = na + group;                            // < NS
    uint32_t ph = 0;
    bool ok = true;
    for (int i0 = group; i0 < n_st && ok; i0 += kGroups * kAhead) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        const int i = i0 + kGroups * d;
        if (i >= n_st || !ok) break;
        // the values first, the wait for their place after
        uint4 v[4];
        const float s0 = FMT == QLORA_NVFP4 ? from_e4m3(sc[d] & 0xFFu) : from_e8m0(sc[d]);
        const float s1 = FMT == QLORA_NVFP4 ? from_e4m3(sc[d] >> 8) : s0;
        v[0] = mx_values8<FMT>(cw[d].x, s0, rs[d]);
        v[1] = mx_values8<FMT>(cw[d].y, s0, rs[d]);
        v[2] = mx_values8<FMT>(cw[d].z, s1, rs[d]);
        v[3] = mx_values8<FMT>(cw[d].w, s1, rs[d]);
        load(i + kGroups * kAhead, d);
        if (lane == 0) ok = wait_after_grid(&S.empty[s], ph ^ 1);
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(S.a[s] + base + ((((q & 1) * 4 + j) ^ (row & 7)) << 4)) = v[j];
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_cluster(mapa_shared(smem_u32(&S.full_a[s]), 0));
          else mbar_arrive(&S.full_a[s]);
        }
        if ((s += kGroups) >= NS) { s -= NS; ph ^= 1; }
      }
    }
  } else {
    grid_dependency_wait();                        // this grid does not end before that kernel
    wait(&S.acc_full, 0);
  }
  __syncwarp();
  if (PAIR && warp == 0 && lane == 0 && *abort) {
    // a wait gave up: the copies in flight count on barriers that may never
    // complete, so give them a millisecond to land
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  const int quad = warp & 3;
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;
  if (PAIR || ls == 0) {
    if (warp >= 2 && warp < 6) {
      tc_fence_after();
      const int e = warp - 2, cw0 = c0 + quad * 32;
      const uint32_t row_off = (uint32_t)((lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4));
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        const int m = m0 + c;
        if (m >= p.M || cw0 >= p.N) break;
        uint32_t v[2][4][4];
        tmem_ld_16x32(tmem + lanes + c, &v[0][0][0]);
        tmem_ld_16x32(tmem + lanes + c + (16u << 16), &v[1][0][0]);
        tmem_wait_ld();
        uint8_t* out = S.out[e][(c >> 5) & 1];
        if (lane == 0) store_wait_read<1>();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = pack_bf16x2(__uint_as_float(v[i >> 1][j][2 * (i & 1)]), __uint_as_float(v[i >> 1][j][2 * (i & 1) + 1]));
          stmatrix_x4_t(smem_u32(out) + row_off + 512 * j, o[0], o[1], o[2], o[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tm_out, out, cw0, m);
          store_commit();
        }
      }
      if (lane == 0) store_wait_read<0>();         // the chunks outlive the stores that read them
    }
  } else {
    cluster_sync();                                // every rank is done with its stages
    const int n = c0 + quad * 32 + lane;
    const bool odd = lane & 1;
    const int live = min(BN, p.M - m0), cs = BN >> ls, lcs = __ffs(cs) - 1;
    float* part = reinterpret_cast<float*>(S.a[0]);
    if (warp >= 2 && warp < 6) {
      tc_fence_after();
      const uint32_t mine = smem_u32(part + rank * cs * 128 + quad * 32 + lane);
#pragma unroll 1
      for (int c = 0; c < live; c += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + lanes + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < live)
            st_cluster_f32(mapa_shared(mine + (uint32_t)(((c + j) & (cs - 1)) * 512), (c + j) >> lcs),
                           __uint_as_float(v[j]));
      }
    }
    cluster_sync();                                // the partial sums have arrived
    if (warp >= 2 && warp < 6) {
      const float* mine = part + quad * 32 + lane;
      const int first = m0 + rank * cs, n_cols = min(cs, p.M - first);
      if (cs >= 8)
        for (int c = 0; c < n_cols; c += 8)
          add_ranks<8, false>(p, mine + c * 128, cs * 128, splits, first + c, n, 1.0f, false, nullptr, 0, odd, true);
      else
        for (int c = 0; c < n_cols; c += 2)
          add_ranks<2, false>(p, mine + c * 128, cs * 128, splits, first + c, n, 1.0f, false, nullptr, 0, odd, true);
    }
  }
  tc_fence_before();
  if (PAIR) cluster_sync();                        // both CTAs done with the paired TMEM
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem, Sh::D_COLS);
    else tmem_dealloc(tmem, Sh::D_COLS);
  }
}

// Expected time in units of 10 ns, and the tile and split that have it: 4 us of
// launch and ramp, the time of a stage and, split, of the reduction.  Fitted on
// B200 to W 4096 x 4096, 18944 x 3584, 3584 x 18944 and 1024 x 1024 with 16 to 1111
// tokens, e.g. W 18944 x 3584: 33 us (16 tokens), 42 (128), 45 (256), 78 (512), 147
// (1111), against 127, 127, 128, 130 and 140 us by way of HBM.
static int64_t cost(int M, int N, int K, int na, int num_sms, int* bn, bool* pair, int* log_splits) {
  constexpr int kShapes = 6;                       // the last: paired SMs
  const int widths[kShapes] = {16, 32, 64, 128, 256, 256}, stage[kShapes] = {38, 38, 40, 46, 50, 46},
            join[kShapes] = {80, 150, 220, 350, 870, 0};
  const int nk = (N + 63) / 64;
  int64_t best = INT64_MAX;
  for (int i = M > 16 ? 1 : 0; i < kShapes; ++i) { // a chunk of output is 32 tokens: 16 only by itself
    const bool two = i == kShapes - 1;
    const int64_t tiles = (two ? (K + 255) / 256 * 2 : (K + 127) / 128) * (int64_t)((M + widths[i] - 1) / widths[i]);
    for (int s = 0; s <= (two ? 0 : 3) && (nk >> s) >= 4; ++s) {
      if (s && (tiles << s) > num_sms + num_sms / 8) break;
      const int64_t waves = s ? 1 : (tiles + num_sms - 1) / num_sms;
      const int64_t c = 400 + waves * (na + (nk + (1 << s) - 1) / (1 << s)) * stage[i] + (s ? join[i] : 0);
      if (c < best) { best = c; *bn = widths[i]; *pair = two; *log_splits = s; }
    }
  }
  return best;
}

// The same of the other way: the weight expanded and transposed to HBM (2.6 bytes
// a weight at 4 TB/s), then the paired-SM GEMM, rounds of 256 x 256 tiles, 0.35 us
// for 64 of the contraction, and 9 us for the launches it adds.
static int64_t cost_expanded(int M, int N, int K, int na, int num_sms) {
  const int64_t tiles = (int64_t)((K + 255) / 256) * ((M + 255) / 256), pairs = std::max(1, num_sms / 2);
  const int64_t rounds = (tiles + pairs - 1) / pairs;
  return 900 + (int64_t)N * K * 26 / 400000 + rounds * (na + (N + 63) / 64) * 35;
}

template <int FMT, int BN, bool PAIR>
static int launch(const qlora_mx_tensor* w, const void* dY, const void* A, int r, const void* sU, int RP, DxArgs g,
                  bool beside, cudaStream_t s) {
  using Sh = Shape<BN, PAIR>;
  CUtensorMap ty, ta, tu, to;
  const int M = g.out.M, K = g.out.N;
  if (!make_tmap_2d_bf16(&ty, dY, g.rows, M, g.rows, 64, Sh::B_ROWS) || !make_tmap_store_bf16(&to, g.out.out, K, M, kChunk))
    return QLORA_ERR_CUDA;
  ta = ty;
  tu = ty;
  if (g.na && (!make_tmap_2d_bf16(&ta, A, K, r, K, 64, 64) || !make_tmap_2d_bf16(&tu, sU, RP, M, RP, 64, Sh::B_ROWS)))
    return QLORA_ERR_CUDA;
  constexpr size_t bytes = sizeof(Smem<BN, PAIR>) + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
  static std::atomic<unsigned long long> attr_devs{0};
  set_smem_attr_once(k_mx_dx<FMT, BN, PAIR>, (int)bytes, attr_devs);
  cudaLaunchConfig_t cfg = {};
  constexpr int cols = 128 * Sh::kCtas;
  cfg.gridDim = dim3((unsigned)((K + cols - 1) / cols * Sh::kCtas) * (unsigned)((M + BN - 1) / BN) << g.log_splits, 1, 1);
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)Sh::kCtas << g.log_splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = beside ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_mx_dx<FMT, BN, PAIR>, ty, ta, tu, to, g) == cudaSuccess ? QLORA_OK : QLORA_ERR_CUDA;
}

template <int FMT>
static int launch_fmt(const qlora_mx_tensor* w, const void* dY, const void* A, int r, const void* sU, int RP, DxArgs g,
                      bool beside, cudaStream_t s, int num_sms) {
  int bn = 0;
  bool pair = false;
  cost(g.out.M, g.rows, g.out.N, g.na, num_sms, &bn, &pair, &g.log_splits);
  if (pair) return launch<FMT, 256, true>(w, dY, A, r, sU, RP, g, beside, s);
  switch (bn) {
    case 16: return launch<FMT, 16, false>(w, dY, A, r, sU, RP, g, beside, s);
    case 32: return launch<FMT, 32, false>(w, dY, A, r, sU, RP, g, beside, s);
    case 64: return launch<FMT, 64, false>(w, dY, A, r, sU, RP, g, beside, s);
    case 128: return launch<FMT, 128, false>(w, dY, A, r, sU, RP, g, beside, s);
    default: return launch<FMT, 256, false>(w, dY, A, r, sU, RP, g, beside, s);
  }
}

}  // namespace dx

bool mx_dx_expands_inside(int M, int N, int K, int na, int num_sms) {
  int bn, ls;
  bool pair;
  return N >= 256 && dx::cost(M, N, K, na, num_sms, &bn, &pair, &ls) <= dx::cost_expanded(M, N, K, na, num_sms);
}

int launch_mx_dx(const qlora_mx_tensor* w, const void* dY, int M, const void* A, int r, const void* sU, int RP, int na,
                 void* dX, bool beside, int* status, cudaStream_t s, int num_sms) {
  dx::DxArgs g{};
  g.out.out = static_cast<__nv_bfloat16*>(dX);
  g.out.M = M;
  g.out.N = (int)w->cols;
  g.packed = w->packed;
  g.scales = w->scales;
  g.row_scale = w->row_scale;
  g.rows = (int)w->rows;
  g.na = na;
  g.status = status;
  return w->format == QLORA_NVFP4 ? dx::launch_fmt<QLORA_NVFP4>(w, dY, A, r, sU, RP, g, beside, s, num_sms)
                                  : dx::launch_fmt<QLORA_MXFP4>(w, dY, A, r, sU, RP, g, beside, s, num_sms);
}

}  // namespace qnf4
