// Microscaled 4-bit floating point: quantise, dequantise, dequantise-transpose.
//
// An element is E2M1 (sign, two exponent bits, one mantissa bit: 0, 0.5, 1,
// 1.5, 2, 3, 4, 6) under a block scale the tensor cores apply themselves:
//   MXFP4  blocks of 32, scale 2^e (E8M0 byte e + 127):
//          e = max(floor(log2 amax) - 2, -127)
//   NVFP4  blocks of 16, scale S (E4M3) under one fp32 scale s per row:
//          s = 2^k, the smallest (k >= -100) with amax_row <= 6 * 448 * s
//          S = E4M3(amax_block / s / 6), nearest, ties to even
//   code = E2M1(x / scale), nearest, ties to even, at most 6 in magnitude.
// All of it is decided exactly.  x / s and x / 2^e are exact (powers of two).
// S has a 4-bit significand, so S times the midpoint of two E2M1 values is
// exact and a quotient x / S that is not on a midpoint differs from it by
// half an fp32 ulp and a fifteenth of it more at least: what is within 2^-28 of
// the real quotient before its rounding to fp32 gets its code.  That is
// q + (y - q S) r for y = x / s, r = RN32(1 / S), q = RN32(y r), one step of
// Newton's method with the residual from one fused multiply-add (on a midpoint
// it gives the midpoint).  28672 x 8192 fp32 163 us; 218 us with a division.
// A bf16 quotient off a midpoint t is off by at least 2^-8 t, so for bf16 input a
// product with RN32(1 / S), rounded to a multiple of 2^-14 (one fused
// multiply-add with 768, one subtraction), decides the same.
//
// W 28672 x 8192 bf16: quantise 84 us MXFP4 (6.8 TB/s), 101 us NVFP4, whose row
// maximum and division of scales make it issue-bound (78 %); dequantise 93 to 98
// us (6.1 TB/s).

#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "mx.h"
#include "mx_values.cuh"
#include "mx_mma.cuh"

namespace qnf4 {

// Eight floats -> eight E2M1 codes, element 0 in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t d;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(d)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return d;
}

// E4M3 byte of a value in [0, 448].
__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(v));
  return d & 0xFFu;
}
constexpr uint32_t kInfBits = 0x7F800000u;

// Consecutive elements of one row that a thread holds, 64 bytes as loaded: 32 of
// bf16, 16 of fp32 (128 bytes a thread took 35 us for 1554 x 18944 fp32, 58 % of
// HBM: the loads of a warp then touch a line each).
template <typename T> struct Unit;
template <> struct Unit<__nv_bfloat16> {
  static constexpr int kElems = 32;
  uint4 w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint32_t word(int j) const {
    const uint4& v = w[j >> 2];
    return (j & 3) == 0 ? v.x : (j & 3) == 1 ? v.y : (j & 3) == 2 ? v.z : v.w;
  }
  // fp32 bits of max |x| over elements [16 h, 16 h + 16); NaN and infinities win
  __device__ __forceinline__ uint32_t amax16(int h) const {
    __nv_bfloat162 m = __habs2(as2(word(8 * h)));
#pragma unroll
    for (int j = 1; j < 8; ++j) m = __hmax2_nan(m, __habs2(as2(word(8 * h + j))));
    const uint32_t b = *reinterpret_cast<const uint32_t*>(&m);
    return max(b << 16, b & 0xFFFF0000u) & 0x7FFFFFFFu;
  }
  __device__ __forceinline__ float value(int i) const {
    return (i & 1) ? bf16_hi(word(i >> 1)) : bf16_lo(word(i >> 1));
  }
  __device__ static __forceinline__ __nv_bfloat162 as2(uint32_t v) {
    return *reinterpret_cast<const __nv_bfloat162*>(&v);
  }
};
template <> struct Unit<float> {
  static constexpr int kElems = 16;
  float4 w[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ float value(int i) const {
    const float4& v = w[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
  __device__ __forceinline__ uint32_t amax16(int h) const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(value(16 * h + i)) & 0x7FFFFFFFu);
    return m;
  }
};

// Codes of elements [16 h, 16 h + 16) of a unit under NVFP4's row factor
// rs = 1 / s and block scale S.
template <typename T>
__device__ __forceinline__ uint2 nv_codes16(const Unit<T>& u, int h, float rs, float S) {
  float v[16];
  const float r = S == 0.0f ? 0.0f : __frcp_rn(S);
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __fadd_rn(__fmaf_rn(u.value(16 * h + i), r * rs, 768.0f), -768.0f);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float y = __fmul_rn(u.value(16 * h + i), rs), q = __fmul_rn(y, r);
      v[i] = __fmaf_rn(__fmaf_rn(-q, S, y), r, q);
    }
  }
  return make_uint2(e2m1x8(v), e2m1x8(v + 8));
}

template <typename T>
__device__ __forceinline__ uint2 mx_codes16(const Unit<T>& u, int h, float inv) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __fmul_rn(u.value(16 * h + i), inv);
  return make_uint2(e2m1x8(v), e2m1x8(v + 8));
}

// One row by nt threads (or by padding, live = false: zero scales only), nt a
// power of two up to 32 or a multiple of 32; every thread of the CTA comes here.
// A thread takes units k = tid + i * nt; with KEEP > 0 (KEEP * nt units at least)
// the row stays in registers between NVFP4's row maximum and the codes, with
// KEEP == 0 it is read twice.  s_max: shared, one word a warp of the row.
template <typename T, int FMT, int KEEP>
__device__ __forceinline__ void quantise_row(const T* __restrict__ x, bool live, int64_t row, int K, int tid, int nt,
                                             uint8_t* __restrict__ packed, uint8_t* __restrict__ scales,
                                             float* __restrict__ row_scale, int* status, uint32_t* s_max) {
  constexpr bool NV = FMT == QLORA_NVFP4;
  constexpr int E = Unit<T>::kElems;
  constexpr int kGroup = 4 * mx_block(FMT) / E;    // units whose scale bytes share a 32-bit word
  const int units = K / E;
  const int upad = (units + kGroup - 1) / kGroup * kGroup;
  const int64_t tiles = mx_scale_tiles(FMT, K);
  Unit<T> u[KEEP > 0 ? KEEP : 1];
  float rs = 1.0f;

  auto emit = [&](int k, const Unit<T>& w) {
    const bool in = live && k < units;
    uint32_t sb = 0;                               // this unit's scale bytes, in their place of the word
    uint2 c[E / 16];
    bool bad = false;
    if constexpr (NV) {
#pragma unroll
      for (int h = 0; h < E / 16; ++h) {
        const uint32_t a = w.amax16(h);
        const bool nf = a >= kInfBits;
        const uint32_t code = to_e4m3(__fdiv_rn(__fmul_rn(__uint_as_float(a), rs), 6.0f));
        c[h] = nv_codes16(w, h, rs, from_e4m3(code));
        if (nf) c[h] = make_uint2(0, 0);
        bad |= nf;
        sb |= (nf ? 0x7Fu : code) << (8 * ((E / 16 * k + h) & 3));
      }
    } else {
      uint32_t a = w.amax16(0);
      if constexpr (E == 32) a = max(a, w.amax16(1));
      else a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));       // the block's other half
      const bool nf = a >= kInfBits;
      const uint32_t code = (uint32_t)max((int)(a >> 23) - 2, 0);
      const float inv = __uint_as_float((254u - code) << 23);
#pragma unroll
      for (int h = 0; h < E / 16; ++h) c[h] = nf ? make_uint2(0, 0) : mx_codes16(w, h, inv);
      bad |= nf;
      const int col = E == 32 ? k : k >> 1;
      if (E == 32 || !(k & 1)) sb = (nf ? 0xFFu : code) << (8 * (col & 3));
    }
    if (!in) sb = 0;
#pragma unroll
    for (int o = 1; o < kGroup; o *= 2) sb |= __shfl_xor_sync(0xFFFFFFFFu, sb, o);
    if (in) {
      uint8_t* out = packed + row * (K / 2) + E / 2 * (int64_t)k;
      if constexpr (E == 32) *reinterpret_cast<uint4*>(out) = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
      else *reinterpret_cast<uint2*>(out) = c[0];
      if (bad) set_status(status, QLORA_ERR_NONFINITE);
    }
    if (k < upad && (k & (kGroup - 1)) == 0)
      *reinterpret_cast<uint32_t*>(scales + mx_scale_offset(row, (int64_t)k * E / mx_block(FMT), tiles)) = sb;
  };
  auto fetch = [&](int k, Unit<T>& w) {
    if (live && k < units) w.load(x + E * (int64_t)k);
    else w.zero();
  };

  if constexpr (KEEP > 0) {
#pragma unroll
    for (int i = 0; i < KEEP; ++i) fetch(tid + i * nt, u[i]);
  }
  if constexpr (NV) {
    uint32_t m = 0;
    auto take = [&](const Unit<T>& v) {
#pragma unroll
      for (int h = 0; h < E / 16; ++h) {
        const uint32_t a = v.amax16(h);
        if (a < kInfBits) m = max(m, a);
      }
    };
    if constexpr (KEEP > 0) {
#pragma unroll
      for (int i = 0; i < KEEP; ++i) take(u[i]);
    } else {
      for (int k = tid; k < units; k += nt) {
        fetch(k, u[0]);
        take(u[0]);
      }
    }
    if (nt >= 32) m = __reduce_max_sync(0xFFFFFFFFu, m);
    else
      for (int o = nt >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (nt > 32) {
      if ((tid & 31) == 0) s_max[tid >> 5] = m;
      __syncthreads();
      m = __reduce_max_sync(0xFFFFFFFFu, (tid & 31) < (nt >> 5) ? s_max[tid & 31] : 0u);
    }
    // s = 2^(f - 127): amax = 1.m 2^E <= 2688 s = 1.3125 * 2^11 s
    uint32_t f = 127;
    if (m) f = (uint32_t)max((int)(m >> 23) - 11 + ((m & 0x7FFFFFu) > 0x280000u ? 1 : 0), 27);
    rs = __uint_as_float((254u - f) << 23);
    if (live && tid == 0) row_scale[row] = __uint_as_float(f << 23);
  }
  if constexpr (KEEP > 0) {
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (i * nt < upad) emit(tid + i * nt, u[i]);
  } else {
    for (int k0 = 0; k0 < upad; k0 += nt) {
      fetch(tid + k0, u[0]);
      emit(tid + k0, u[0]);
    }
  }
}

// blockDim.x threads a row, blockDim.y rows a CTA (one if a row has several warps).
template <typename T, int FMT, int KEEP>
__global__ void __launch_bounds__(512)
k_mx_quantize(const T* __restrict__ X, int64_t ld, int rows, int K, uint8_t* __restrict__ packed,
              uint8_t* __restrict__ scales, float* __restrict__ row_scale, int* status) {
  __shared__ uint32_t s_max[16];
  grid_launch_dependents();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;   // rows past the last write the padding's zero scales
  quantise_row<T, FMT, KEEP>(X + row * ld, row < rows, row, K, threadIdx.x, blockDim.x, packed, scales, row_scale,
                             status, s_max);
  // beside the kernel before it, this grid does not end before that one: what waits
  // for this grid waits for both
  if (blockIdx.x == gridDim.x - 1) grid_dependency_wait();
}

// Threads and rows of a CTA: a unit a thread up to 256 units, several rows a CTA
// when they are short (a CTA a row: 400000 x 64 bf16 took 419 us).
template <typename T, int FMT>
static void launch_mx_quantize_t(const void* X, int64_t rows, int64_t cols, int64_t ld, uint8_t* packed,
                                 uint8_t* scales, float* row_scale, bool beside, int* status, cudaStream_t s) {
  constexpr int E = Unit<T>::kElems;
  constexpr int kGroup = 4 * mx_block(FMT) / E;
  const int units = (int)(cols / E);
  const int upad = (units + kGroup - 1) / kGroup * kGroup;
  const int64_t prow = (rows + 127) / 128 * 128;
  auto run = [&](auto kern, int per) {
    const int rounds = std::max(per, (upad + 511) / 512);          // equal rounds of at most 512 threads
    int nt = ((upad + rounds - 1) / rounds + 31) / 32 * 32, group = 1;
    if (upad <= 16) {
      nt = kGroup;
      while (nt < upad) nt *= 2;
    }
    while (nt <= 32 && group * nt < 256) group *= 2;               // at most 128: divides prow
    launch_dependent(kern, dim3((unsigned)(prow / group)), dim3(nt, group), beside, s, (const T*)X, ld, (int)rows, (int)cols,
                     packed, scales, row_scale, status);
  };
  if constexpr (FMT != QLORA_NVFP4) run(k_mx_quantize<T, FMT, 0>, 1);
  else if (upad <= 256) run(k_mx_quantize<T, FMT, 1>, 1);
  else if (upad <= 1024) run(k_mx_quantize<T, FMT, 2>, 2);
  else if (upad <= 1536) run(k_mx_quantize<T, FMT, 3>, 3);
  else run(k_mx_quantize<T, FMT, 0>, 1);
}

void launch_mx_quantize(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, int format,
                        uint8_t* packed, uint8_t* scales, float* row_scale, bool beside, int* status,
                        cudaStream_t s) {
  if (dtype == QLORA_F32) {
    if (format == QLORA_NVFP4) launch_mx_quantize_t<float, QLORA_NVFP4>(X, rows, cols, ld, packed, scales, row_scale, beside, status, s);
    else launch_mx_quantize_t<float, QLORA_MXFP4>(X, rows, cols, ld, packed, scales, row_scale, beside, status, s);
  } else {
    if (format == QLORA_NVFP4) launch_mx_quantize_t<__nv_bfloat16, QLORA_NVFP4>(X, rows, cols, ld, packed, scales, row_scale, beside, status, s);
    else launch_mx_quantize_t<__nv_bfloat16, QLORA_MXFP4>(X, rows, cols, ld, packed, scales, row_scale, beside, status, s);
  }
}

// ===========================================================================
// What the layer does with few tokens before its product, in one launch: the
// tokens quantised, a CTA a row, and T = X A^T.  A cluster takes eight rows of A
// and cuts the contraction in 64 slices, one a warp (mma.m16n8k16 on 16-byte
// words straight from global memory: a lane's words of X and A hold the same
// eight k, so their order within the product does not matter); the warps' sums
// are added in order, in the CTA and then by rank 0.  The product may start
// meanwhile: it reads the weight first and waits for this grid before anything
// written here.
// ===========================================================================
template <int FMT, int MT>
__global__ void __cluster_dims__(8, 1, 1) __launch_bounds__(256)
k_mx_prep(const __nv_bfloat16* __restrict__ X, int M, int K, const __nv_bfloat16* __restrict__ A, int r,
          uint8_t* __restrict__ packed, uint8_t* __restrict__ scales, float* __restrict__ row_scale, float s,
          __nv_bfloat16* __restrict__ sT, __nv_bfloat16* __restrict__ T_save, int* status) {
  __shared__ uint32_t s_max[16];
  __shared__ float s_warp[8][MT * 8];              // [warp][token * 8 + row of A]
  __shared__ float s_rank[8][MT * 8];              // rank 0: the ranks' sums
  grid_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((int)blockIdx.x >= r) {
    const int row = (int)blockIdx.x - r;
    if (row < M)
      quantise_row<__nv_bfloat16, FMT, 3>(X + (int64_t)row * K, true, row, K, tid, 256, packed, scales, row_scale,
                                          status, s_max);
    return;                                        // whole clusters: r is a multiple of 8
  }
  const int rank = (int)cluster_ctarank();
  const int j0 = (int)blockIdx.x & ~7;
  const int g = lane >> 2, t = lane & 3;
  const int steps = K / 32, slice = rank * 8 + warp;
  const int k0 = steps * slice / 64, k1 = steps * (slice + 1) / 64;
  const __nv_bfloat16* a = A + (int64_t)(j0 + g) * K + 8 * t;
  const __nv_bfloat16* x = X + (int64_t)g * K + 8 * t;
  float acc[MT / 16][4];
#pragma unroll
  for (int i = 0; i < MT / 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
#pragma unroll 4
  for (int k = k0; k < k1; ++k) {
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(a + 32 * (int64_t)k));
    uint4 v[MT / 8];
#pragma unroll
    for (int i = 0; i < MT / 8; ++i)
      v[i] = 8 * i + g < M ? __ldg(reinterpret_cast<const uint4*>(x + (int64_t)(8 * i) * K + 32 * (int64_t)k))
                           : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < MT / 16; ++i) {
      mma_16816(acc[i], v[2 * i].x, v[2 * i + 1].x, v[2 * i].y, v[2 * i + 1].y, b.x, b.y);
      mma_16816(acc[i], v[2 * i].z, v[2 * i + 1].z, v[2 * i].w, v[2 * i + 1].w, b.z, b.w);
    }
  }
#pragma unroll
  for (int i = 0; i < MT / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)                    // token g or g + 8, row 2 t or 2 t + 1 of A
      s_warp[warp][(16 * i + g + 8 * (e >> 1)) * 8 + 2 * t + (e & 1)] = acc[i][e];
  cluster_sync();                                  // s_warp is whole, rank 0 runs
  for (int i = tid; i < MT * 8; i += 256) {
    float sum = s_warp[0][i];
#pragma unroll
    for (int w = 1; w < 8; ++w) sum = __fadd_rn(sum, s_warp[w][i]);
    asm volatile("st.shared::cluster.f32 [%0], %1;"
                 :: "r"(mapa_shared(smem_u32(&s_rank[rank][i]), 0)), "f"(sum) : "memory");
  }
  cluster_sync();
  if (rank == 0)
    for (int i = tid; i < M * 8; i += 256) {
      float sum = s_rank[0][i];
#pragma unroll
      for (int z = 1; z < 8; ++z) sum = __fadd_rn(sum, s_rank[z][i]);
      const int64_t at = (int64_t)(i >> 3) * r + j0 + (i & 7);
      sT[at] = __float2bfloat16_rn(__fmul_rn(s, sum));
      if (T_save) T_save[at] = __float2bfloat16_rn(sum);
    }
}

void launch_mx_prep(const void* X, int M, int K, const void* A, int r, int format, uint8_t* packed, uint8_t* scales,
                    float* row_scale, float s, void* sT, void* T_save, int* status, cudaStream_t st) {
  const unsigned grid = (unsigned)(r + (M + 7) / 8 * 8);
  auto run = [&](auto kern) {
    kern<<<grid, 256, 0, st>>>((const __nv_bfloat16*)X, M, K, (const __nv_bfloat16*)A, r, packed, scales, row_scale, s,
                               (__nv_bfloat16*)sT, (__nv_bfloat16*)T_save, status);
  };
  if (format == QLORA_NVFP4) {
    if (M <= 16) run(k_mx_prep<QLORA_NVFP4, 16>);
    else if (M <= 32) run(k_mx_prep<QLORA_NVFP4, 32>);
    else run(k_mx_prep<QLORA_NVFP4, 64>);
  } else {
    if (M <= 16) run(k_mx_prep<QLORA_MXFP4, 16>);
    else if (M <= 32) run(k_mx_prep<QLORA_MXFP4, 32>);
    else run(k_mx_prep<QLORA_MXFP4, 64>);
  }
}

// ===========================================================================
// Dequantise: value = RNbf16(RN32(q S s)).  q S is exact (2 + 4 significant
// bits), and so is the bf16 result when s is a power of two, as the quantiser
// writes it.  Eight elements a thread and step: a 4-byte code word, a 16-byte
// store.  blockDim.x threads share a row, blockDim.y rows a CTA, about eight words
// a thread (18944 x 3584: 32.6 us, 38.8 us with two).
// ===========================================================================
template <int FMT>
__global__ void __launch_bounds__(256)
k_mx_dequantize(const uint8_t* __restrict__ packed, const uint8_t* __restrict__ scales,
                const float* __restrict__ row_scale, int rows, int K, __nv_bfloat16* __restrict__ out) {
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= rows) return;
  const int64_t tiles = mx_scale_tiles(FMT, K);
  const float rs = FMT == QLORA_NVFP4 ? row_scale[row] : 1.0f;
  const uint32_t* c = reinterpret_cast<const uint32_t*>(packed + row * (K / 2));
  uint4* o = reinterpret_cast<uint4*>(out + row * K);
  const uint8_t* sc = scales + mx_scale_offset(row, 0, tiles);
  const int words = K / 8;
#pragma unroll 4
  for (int w = threadIdx.x; w < words; w += blockDim.x) {
    const int col = w / (mx_block(FMT) / 8);
    __stcs(o + w, mx_values8<FMT>(__ldg(c + w), mx_scale_value<FMT>(__ldg(sc + (int64_t)(col >> 2) * 512 + (col & 3))), rs));
  }
}

void launch_mx_dequantize(const qlora_mx_tensor* t, void* out, cudaStream_t s) {
  int tx = 8;                                      // about eight words a thread
  while (tx < 256 && 8 * tx < t->cols / 8) tx *= 2;
  const dim3 block(tx, 256 / tx);
  const unsigned grid = (unsigned)((t->rows + block.y - 1) / block.y);
  auto run = [&](auto kern) {
    kern<<<grid, block, 0, s>>>(t->packed, t->scales, t->row_scale, (int)t->rows, (int)t->cols, (__nv_bfloat16*)out);
  };
  if (t->format == QLORA_NVFP4) run(k_mx_dequantize<QLORA_NVFP4>);
  else run(k_mx_dequantize<QLORA_MXFP4>);
}

// ===========================================================================
// Dequantise-transpose for the backward's dX: CTA tile 64 rows (n) x 256 columns
// (k), bound by the 2-byte stores.  Thread (pr, qk) expands rows 2 pr, 2 pr + 1,
// columns [32 qk, 32 qk + 32) from 16-byte words and stores each column's pair of
// rows as one word of the transposed tile in shared memory (a warp's words are
// consecutive); the tile leaves in 16-byte stores, 128 bytes a row.
// ===========================================================================
template <int FMT>
__global__ void __launch_bounds__(256)
k_mx_dequant_t(const uint8_t* __restrict__ packed, const uint8_t* __restrict__ scales,
               const float* __restrict__ row_scale, int N, int K, __nv_bfloat16* __restrict__ Wt) {
  constexpr int kPitch = 36;                       // words per transposed row (32 + pad, 16-byte rows)
  __shared__ __align__(16) uint32_t tileT[256 * kPitch];
  const unsigned tiles_k = (unsigned)(K + 255) / 256;
  const int n0 = (int)(blockIdx.x / tiles_k) * 64, k0 = (int)(blockIdx.x % tiles_k) * 256;
  const int tid = threadIdx.x;
  const int pr = tid & 31, qk = tid >> 5;
  const int k = k0 + 32 * qk;
  const int64_t tiles = mx_scale_tiles(FMT, K);
  uint4 cw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  float S[2][2] = {}, rs[2] = {1.0f, 1.0f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = n0 + 2 * pr + h;
    if (k < K && n < N) {                          // K % 32 == 0: 32 columns or none
      cw[h] = __ldg(reinterpret_cast<const uint4*>(packed + ((int64_t)n * K + k) / 2));
      if (FMT == QLORA_NVFP4) {
        const uint32_t b = *reinterpret_cast<const uint16_t*>(scales + mx_scale_offset(n, k / 16, tiles));
        S[h][0] = from_e4m3(b & 0xFFu);
        S[h][1] = from_e4m3(b >> 8);
        rs[h] = row_scale[n];
      } else {
        S[h][0] = S[h][1] = from_e8m0(scales[mx_scale_offset(n, k / 32, tiles)]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint4 v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[h] = mx_values8<FMT>(q == 0 ? cw[h].x : q == 1 ? cw[h].y : q == 2 ? cw[h].z : cw[h].w, S[h][q >> 1], rs[h]);
    const uint32_t a[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, b[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t* t = tileT + (32 * qk + 8 * q + 2 * j) * kPitch + pr;
      t[0] = prmt(a[j], b[j], 0x5410);
      t[kPitch] = prmt(a[j], b[j], 0x7632);
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int i = tid; i < 256 * 8; i += 256) {
    const int kr = i >> 3, ch = i & 7;             // transposed row, 16-byte chunk (8 columns n)
    const int kk = k0 + kr, nn = n0 + ch * 8;
    if (kk < K && nn < N)                          // N % 8 == 0: a chunk is whole
      *reinterpret_cast<uint4*>(Wt + (int64_t)kk * N + nn) =
          *reinterpret_cast<const uint4*>(&tileT[kr * kPitch + ch * 4]);
  }
  if (blockIdx.x == gridDim.x - 1) grid_dependency_wait();         // ends after the kernel it runs beside
}

void launch_mx_dequant_t(const qlora_mx_tensor* w, void* Wt, bool beside, cudaStream_t s) {
  const unsigned grid = (unsigned)((w->cols + 255) / 256) * (unsigned)((w->rows + 63) / 64);
  auto run = [&](auto kern) {
    launch_dependent(kern, dim3(grid), dim3(256), beside, s, w->packed, w->scales, w->row_scale, (int)w->rows, (int)w->cols,
                     (__nv_bfloat16*)Wt);
  };
  if (w->format == QLORA_NVFP4) run(k_mx_dequant_t<QLORA_NVFP4>);
  else run(k_mx_dequant_t<QLORA_MXFP4>);
}

// ===========================================================================
// Adapter factors for the product: zero-padded to RP columns and, for NVFP4,
// divided by the row scale that the product's epilogue multiplies back.  The
// quantiser's row scales are powers of two, for which this is exact; any
// other row scale costs one more bf16 rounding of the factor.
// ===========================================================================
__global__ void __launch_bounds__(256)
k_mx_pad_rows(const __nv_bfloat16* in, int64_t rows, int r, int ldi, int RP, const float* __restrict__ row_scale,
              __nv_bfloat16* out) {
  grid_launch_dependents();
  const int per = RP / 8;                          // 16-byte words of an output row (8 or 16)
  const int64_t total = rows * per;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = per == 8 ? i >> 3 : i >> 4;
    const int c = 8 * (int)(i & (per - 1));
    uint4 v = make_uint4(0, 0, 0, 0);
    if (c < r) v = *reinterpret_cast<const uint4*>(in + row * ldi + c);
    if (row_scale) {
      const float s = row_scale[row];
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(__fdiv_rn(bf16_lo(w[j]), s), __fdiv_rn(bf16_hi(w[j]), s));
    }
    *reinterpret_cast<uint4*>(out + row * RP + c) = v;
  }
}

void launch_mx_pad_rows(const void* in, int64_t rows, int r, int ldi, int RP, const float* row_scale,
                        void* out, cudaStream_t s) {
  const int grid = (int)std::min<int64_t>((rows * (RP / 8) + 255) / 256, 148 * 8);
  k_mx_pad_rows<<<grid, 256, 0, s>>>((const __nv_bfloat16*)in, rows, r, ldi, RP, row_scale, (__nv_bfloat16*)out);
}

}  // namespace qnf4
