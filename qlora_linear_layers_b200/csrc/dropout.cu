// Dropout as an operator of its own: the mask of the layer's adapter dropout
// (Philox4x64-10, one block for eight elements; common.cuh) regenerated
// wherever it is needed and never stored.
//
//   forward   Y  = RN(RN32(D c X) + R)      backward   dX = RN(RN32(D c dY))
//
// D keeps element e = first + row * cols + col.  Bytes: each input read once,
// the output written once; the generator costs 18 64 x 64-bit products a
// block, which is what bounds bf16 tensors (8192 x 3584: 48 us, with a residual 49
// us; the bytes alone 18 and 27 us).

#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "draw.cuh"

namespace qnf4 {

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// The general kernel, element by element (8192 x 3584 from number 1: 108 us bf16, 142 us
// fp32, against 45 and 46 us of the one below): any width, strides and first number.  One thread a
// Philox block: elements 8 blk .. 8 blk + 7 of the numbering that starts at 0,
// of which [first, first + rows * cols) exist here.
template <typename T>
__global__ void __launch_bounds__(256)
k_dropout(const T* X, int64_t ldx, const T* R, int64_t ldr, T* Y, int64_t ldy, int64_t n, int64_t cols,
          int64_t first, const __grid_constant__ DropoutKeys d) {
  const int64_t b0 = first >> 3, b1 = (first + n + 7) >> 3;
  for (int64_t blk = b0 + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; blk < b1;
       blk += (int64_t)gridDim.x * blockDim.x) {
    const Draw draw = draw8((uint64_t)blk, d);
    uint32_t keep = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) keep |= draw.keep(i, d.thr8) ? 1u << i : 0u;
    // row and column of the block's first element here; they advance from there
    const int64_t e0 = max((int64_t)0, blk * 8 - first), e1 = min(n, blk * 8 + 8 - first);
    int64_t row = (e0 | cols) >> 32 ? e0 / cols : (int64_t)((uint32_t)e0 / (uint32_t)cols);
    int64_t col = e0 - row * cols;
    const int shift = (int)(first + e0 - blk * 8);
    T x[8], r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (e0 + i < e1) {
        x[i] = X[row * ldx + col];
        if (R) r[i] = R[row * ldr + col];
        if (++col == cols) { col = 0; ++row; }
      }
    }
    row = (e0 | cols) >> 32 ? e0 / cols : (int64_t)((uint32_t)e0 / (uint32_t)cols);
    col = e0 - row * cols;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (e0 + i < e1) {
        float v = (keep >> (shift + i)) & 1u ? __fmul_rn(to_f32(x[i]), d.scale) : 0.0f;
        if (R) v = __fadd_rn(v, to_f32(r[i]));
        Y[row * ldy + col] = from_f32<T>(v);
        if (++col == cols) { col = 0; ++row; }
      }
    }
  }
}

// Eight elements of a row from 16-byte words, once a block lies in one row and
// on its own 16-byte boundary: cols, strides and first multiples of 8.
template <typename T> struct Oct;
template <> struct Oct<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { v[2 * j] = bf16_lo(w[j]); v[2 * j + 1] = bf16_hi(w[j]); }
  }
  __device__ __forceinline__ void set(const float* v) {
    a = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};
template <> struct Oct<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float* v) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// kUnroll blocks a thread and step, a grid-stride apart, so that one block's
// loads and products cover the other's latencies.  DENSE: rows without gaps, one
// index for all operands, and a last block of `tail` elements.
constexpr int kUnroll = 2;
template <typename T, bool RES, bool DENSE>
__global__ void __launch_bounds__(256)
k_dropout8(const T* X, int64_t ldx, const T* R, int64_t ldr, T* Y, int64_t ldy, int64_t blocks, int64_t row_blocks,
           int tail, int64_t first_block, const __grid_constant__ DropoutKeys d) {
  grid_launch_dependents();
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t b = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; b < blocks; b += kUnroll * step) {
    Oct<T> x[kUnroll], r[kUnroll];
    int64_t row[kUnroll], col[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int64_t k = b + i * step;
      row[i] = 0;
      col[i] = 8 * k;
      if (!DENSE) {
        row[i] = k / row_blocks;
        col[i] = 8 * (k - row[i] * row_blocks);
      }
      if (i == 0 || k < blocks) {
        x[i].load(X + row[i] * ldx + col[i]);
        if (RES) r[i].load(R + row[i] * ldr + col[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const Draw draw = draw8((uint64_t)(first_block + b + i * step), d);
      float v[8], w[8];
      x[i].get(v);
      if (RES) r[i].get(w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = draw.keep(j, d.thr8) ? __fmul_rn(v[j], d.scale) : 0.0f;
        if (RES) v[j] = __fadd_rn(v[j], w[j]);
      }
      x[i].set(v);
      if (i == 0 || b + i * step < blocks) x[i].store(Y + row[i] * ldy + col[i]);
    }
  }
  if (DENSE && tail && blockIdx.x == gridDim.x - 1 && threadIdx.x < tail) {
    const int j = threadIdx.x;
    const int64_t e = 8 * blocks + j;
    const Draw draw = draw8((uint64_t)(first_block + blocks), d);
    bool keep = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) keep = i == j ? draw.keep(i, d.thr8) : keep;
    float v = keep ? __fmul_rn(to_f32(X[e]), d.scale) : 0.0f;
    if (RES) v = __fadd_rn(v, to_f32(R[e]));
    Y[e] = from_f32<T>(v);
  }
}

template <typename T>
static void launch_dropout_t(const T* X, int64_t ldx, const T* R, int64_t ldr, T* Y, int64_t ldy, int64_t rows,
                             int64_t cols, int64_t first, const Dropout& drop, int per_sm, cudaStream_t s) {
  const DropoutKeys d = make_keys(drop);
  const int64_t n = rows * cols;
  const int64_t blocks = (n + 14) / 8;
  const bool dense = (ldx == cols && ldy == cols && (!R || ldr == cols)) || rows == 1;
  if (first % 8 == 0 && (dense || (cols | ldx | ldy | (R ? ldr : 0)) % 8 == 0)) {
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((n / 8 + 511) / 512, 148 * per_sm));
    auto run = [&](auto kern) {
      kern<<<grid, 256, 0, s>>>(X, ldx, R, ldr, Y, ldy, n / 8, cols / 8, (int)(n % 8), first / 8, d);
    };
    if (R) {
      if (dense) run(k_dropout8<T, true, true>);
      else run(k_dropout8<T, true, false>);
    } else {
      if (dense) run(k_dropout8<T, false, true>);
      else run(k_dropout8<T, false, false>);
    }
    return;
  }
  const unsigned grid = (unsigned)std::min<int64_t>((blocks + 255) / 256, 148 * 8);
  k_dropout<T><<<grid, 256, 0, s>>>(X, ldx, R, ldr, Y, ldy, n, cols, first, d);
}

void launch_dropout(const void* X, int64_t ldx, const void* R, int64_t ldr, void* Y, int64_t ldy, int dtype,
                    int64_t rows, int64_t cols, int64_t first, const Dropout& d, cudaStream_t s, int per_sm) {
  if (dtype == QLORA_F32)
    launch_dropout_t((const float*)X, ldx, (const float*)R, ldr, (float*)Y, ldy, rows, cols, first, d, per_sm, s);
  else
    launch_dropout_t((const __nv_bfloat16*)X, ldx, (const __nv_bfloat16*)R, ldr, (__nv_bfloat16*)Y, ldy, rows, cols,
                     first, d, per_sm, s);
}

}  // namespace qnf4
