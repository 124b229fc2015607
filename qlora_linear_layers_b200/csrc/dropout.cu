// Dropout as an operator of its own: the mask of the layer's adapter dropout
// (Philox4x64-10, one block for eight elements; common.cuh) regenerated
// wherever it is needed and never stored.
//
//   forward   Y  = RN(RN32(D c X) + R)      backward   dX = RN(RN32(D c dY))
//
// D keeps element e = first + row * cols + col.  Bytes: each input read once,
// the output written once; the generator costs twenty 64 x 64-bit products a
// block, which is what bounds bf16 tensors.

#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace qnf4 {

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// One thread a Philox block: elements 8 blk .. 8 blk + 7 of the numbering that
// starts at 0, of which [first, first + rows * cols) exist here.
template <typename T>
__global__ void __launch_bounds__(256)
k_dropout(const T* X, int64_t ldx, const T* R, int64_t ldr, T* Y, int64_t ldy, int64_t n, int64_t cols,
          int64_t first, Dropout d) {
  const int64_t b0 = first >> 3, b1 = (first + n + 7) >> 3;
  for (int64_t blk = b0 + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; blk < b1;
       blk += (int64_t)gridDim.x * blockDim.x) {
    const uint32_t keep = d.on ? dropout_keep8((uint64_t)blk, d.seed, d.thr) : 0xFFu;
    for (int i = 0; i < 8; ++i) {
      const int64_t e = blk * 8 + i - first;
      if (e < 0 || e >= n) continue;
      const int64_t row = e / cols, col = e - row * cols;
      float v = (keep >> i) & 1u ? __fmul_rn(to_f32(X[row * ldx + col]), d.scale) : 0.0f;
      if (R) v = __fadd_rn(v, to_f32(R[row * ldr + col]));
      Y[row * ldy + col] = from_f32<T>(v);
    }
  }
}

void launch_dropout(const void* X, int64_t ldx, const void* R, int64_t ldr, void* Y, int64_t ldy, int dtype,
                    int64_t rows, int64_t cols, int64_t first, const Dropout& d, cudaStream_t s) {
  const int64_t blocks = (rows * cols + 14) / 8;
  const unsigned grid = (unsigned)std::min<int64_t>((blocks + 255) / 256, 148 * 8);
  if (dtype == QLORA_F32)
    k_dropout<float><<<grid, 256, 0, s>>>((const float*)X, ldx, (const float*)R, ldr, (float*)Y, ldy, rows * cols,
                                          cols, first, d);
  else
    k_dropout<__nv_bfloat16><<<grid, 256, 0, s>>>((const __nv_bfloat16*)X, ldx, (const __nv_bfloat16*)R, ldr,
                                                  (__nv_bfloat16*)Y, ldy, rows * cols, cols, first, d);
}

}  // namespace qnf4
