// Pieces that the kernels of the microscaled product share.
//
// Tensor memory: kernels of two streams may meet on an SM, and a CTA that waits
// for columns while its cluster's other CTAs hold theirs must not wait for one that
// waits for it.  None has to wait: any kernels of this library that fit an SM
// together by their shared memory need at most 512 columns together (a product's
// two CTAs 256 each, the adapter's 128 or 256 each; the paired kernels leave no room).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "gemm.h"
#include "mx.h"

namespace qnf4 {
namespace mx {

constexpr int BW = 128;                            // weight rows of a CTA's tile
constexpr int BKB = 128;                           // bytes of a row and stage: 256 codes or 64 bf16

struct Args {
  const float* xr;          // row scales (NVFP4)
  const float* wr;
  __nv_bfloat16* out;
  int M, N, K;
  int na;                   // adapter K steps
  int r;                    // rank of the adapter added by the epilogue, 0: none
  const __nv_bfloat16* sT;  // [M, r]
  const __nv_bfloat16* B;   // [N, r]
  int* status;
};

// mx_gemm_pair.cu
int64_t pair_cost(const Args& a, int num_sms);
int pair_rounds(const Args& a, int num_sms);
int launch_gemm_pair(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const MxAdapter& ad, bool after_prep,
                     const Args& a, cudaStream_t s, int num_sms);

constexpr int kFewTokens = 32;                     // up to here the kernel for few tokens

// Barrier of `Threads` threads; true if any of them came with true.
template <int Id, int Threads>
__device__ __forceinline__ bool barrier_or(bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any) : "r"((uint32_t)v), "n"(Id), "n"(Threads) : "memory");
  return any != 0;
}

// True in one lane of a converged warp.  The tensor-core and TMA instructions
// take their operands from uniform registers; behind an elect.sync the compiler
// knows that one lane is active and issues them directly, behind a comparison of
// the lane number it loops over the lanes (measured: 154 against 45 cycles of
// issue for an MMA, 73 against 32 for a scale copy).
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// Tensor map of a scale array: 512-byte tiles, tiles along K, 128-row blocks;
// boxes of nt x rb tiles.  Tiles past the array read as zero.
inline bool make_scale_tmap(CUtensorMap* tm, const uint8_t* scales, int format, int64_t rows, int64_t cols,
                            uint32_t nt, uint32_t rb) {
  const uint64_t tiles = (uint64_t)mx_scale_tiles(format, cols);
  const uint64_t dims[3] = {256, tiles, (uint64_t)((rows + 127) / 128)};
  const uint64_t strides[2] = {512, tiles * 512};
  const uint32_t box[3] = {256, nt, rb};
  return make_tmap_3d(tm, scales, true, dims, strides, box, false);
}

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

// 512-byte scale tile in shared memory: 32 rows of 16 bytes, no swizzle,
// groups of eight rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFFu);
  d |= (uint64_t)(128u >> 4) << 16;
  d |= (uint64_t)(128u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  return d;
}

// Scale tile -> four tensor-memory columns, replicated to the four lane groups.
__device__ __forceinline__ void scale_copy(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void scale_copy_pair(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of the 4-bit block-scaled kinds: A = B = E2M1, both
// K-major, K = 64; sf is the byte of a scale word where this K step begins
// (0, or 2 in the second half of an MXFP4 word).
template <int FMT>
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((FMT == QLORA_MXFP4 ? 1u : 0u) << 23) | ((uint32_t)(M >> 7) << 27) | (sf << 29);
}

#define QNF4_MMA_MX(NAME, GROUP)                                                                             \
  template <int FMT>                                                                                         \
  __device__ __forceinline__ void NAME(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,     \
                                       uint32_t sfb, uint32_t accumulate) {                                  \
    if constexpr (FMT == QLORA_NVFP4)                                                                        \
      asm volatile(                                                                                          \
          "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                  \
          "tcgen05.mma." GROUP ".kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" \
          :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");            \
    else                                                                                                     \
      asm volatile(                                                                                          \
          "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                  \
          "tcgen05.mma." GROUP ".kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" \
          :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");            \
  }
QNF4_MMA_MX(mma_mx, "cta_group::1")
QNF4_MMA_MX(mma_mx_pair, "cta_group::2")
#undef QNF4_MMA_MX

// Tiled 3-D load into this CTA's shared memory whose completion is counted on
// an mbarrier of either CTA of the pair (no multicast).
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const void* tmap, uint32_t mbar_cluster,
                                                 int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];"
      :: "r"(smem_u32(smem_dst)), "l"(tmap), "r"(mbar_cluster), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

constexpr int kChunk = 32;                         // tokens of an output chunk

// Warp-wide: 16 lanes x 32 columns of tensor memory; of every 8 columns thread t
// gets columns 2 (t % 4), + 1 of lane t / 4 (v[4 j], v[4 j + 1]) and of lane
// t / 4 + 8 (v[4 j + 2], v[4 j + 3]).
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// Four 8 x 8 bf16 blocks of a warp, transposed: row i of block j goes to the
// address that lane 8 j + i holds.
__device__ __forceinline__ void stmatrix_x4_t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
               :: "r"(addr), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}

__device__ __forceinline__ void tma_store_2d(const void* tmap, const void* smem_src, int32_t c0, int32_t c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
               :: "l"(tmap), "r"(smem_u32(smem_src)), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" :: "n"(N) : "memory");
}


// A sum times its two row scales.  Their product is formed first, one multiplication
// for both and exact for powers of two, where it is a normal number; scales far from 1
// (`far`) may have a product that is not, although the result is: then the larger one
// comes first, so that the sum is moved out of range only if the result is.
__device__ __forceinline__ bool scale_far(float s) { return !(s >= 0x1p-62f && s <= 0x1p62f); }
__device__ __forceinline__ float times_scales(float x, float rx, float rw, bool far) {
  const float s = __fmul_rn(rx, rw);
  if (far && !(s >= 0x1p-126f && s <= 0x1.fffffep127f))
    return rx > rw ? __fmul_rn(__fmul_rn(x, rx), rw) : __fmul_rn(__fmul_rn(x, rw), rx);
  return __fmul_rn(x, s);
}

// Store into another CTA of the cluster (address from mapa_shared).
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(addr), "f"(v) : "memory");
}

// Bounded wait for a copy in flight after the kernel has given up (the abort
// flag is set and no longer looked at).
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, const int* st) {
  const uint64_t t0 = globaltimer_ns(), lim = wait_limit_ns(st);
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < lim) {
  }
}

// A lane's NC results (tokens m .. m + NC - 1 of output column n) -> bf16 rows.
// With an even N lanes (2i, 2i + 1) swap halves: even lanes store tokens m + j,
// odd lanes m + j + 1, both the two outputs at `col`, the even lane's column.
template <int NC>
__device__ __forceinline__ void store_columns(const Args& p, const uint32_t* v, int m, int n, int col, bool odd,
                                              bool pairs) {
  if (pairs) {
    const int first = m + (odd ? 1 : 0);
    const int left = col < p.N ? p.M - first : 0;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (int64_t)first * p.N + col);
#pragma unroll
    for (int j = 0; j < NC; j += 2) {
      const uint32_t mine = pack_bf16x2(__uint_as_float(v[j]), __uint_as_float(v[j + 1]));
      const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, mine, 1);
      const uint32_t o = odd ? prmt(other, mine, 0x7632) : prmt(mine, other, 0x5410);
      if (j < left) *dst = o;
      dst += p.N;                                  // two bf16 rows = N words
    }
  } else {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (m + j < p.M && n < p.N) p.out[(int64_t)(m + j) * p.N + n] = __float2bfloat16_rn(__uint_as_float(v[j]));
  }
}

// Add the ranks' partial sums of NC token columns (in rank order), scale, store.
template <int NC, bool NV>
__device__ __forceinline__ void add_ranks(const Args& p, const float* part, int rank_stride, int splits, int m, int n,
                                          float rw, bool far, const float* add, int add_pitch, bool odd, bool pairs) {
  float sum[NC], rx[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) rx[j] = NV && m + j < p.M ? p.xr[m + j] : 0.0f;
#pragma unroll
  for (int j = 0; j < NC; ++j) sum[j] = part[j * 128];
  for (int z = 1; z < splits; ++z)
#pragma unroll
    for (int j = 0; j < NC; ++j) sum[j] = __fadd_rn(sum[j], part[z * rank_stride + j * 128]);
  uint32_t v[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if (NV) sum[j] = times_scales(sum[j], rx[j], rw, far);
    if (add) sum[j] = __fadd_rn(sum[j], add[j * add_pitch]);
    v[j] = __float_as_uint(sum[j]);
  }
  store_columns<NC>(p, v, m, n, n - (odd ? 1 : 0), odd, pairs);
}

}  // namespace mx
}  // namespace qnf4
