// Launchers of the microscaled 4-bit kernels (mx_quant.cu, mx_gemm.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/qlora_nf4.h"

namespace qnf4 {

// Block of a format: elements that share one scale byte.
__host__ __device__ constexpr int mx_block(int format) { return format == QLORA_NVFP4 ? 16 : 32; }

// Scale tiles (128 rows x 4 scale columns, 512 bytes) along a row of `cols`
// elements; one tile spans 64 (NVFP4) or 128 (MXFP4) elements.
__host__ __device__ constexpr int64_t mx_scale_tiles(int format, int64_t cols) {
  return (cols + 4 * mx_block(format) - 1) / (4 * mx_block(format));
}

// Byte of scale (row r, scale column c) in the tiled array.
__host__ __device__ constexpr int64_t mx_scale_offset(int64_t r, int64_t c, int64_t tiles) {
  return ((r >> 7) * tiles + (c >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (c & 3);
}

void launch_mx_quantize(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, int format,
                        uint8_t* packed, uint8_t* scales, float* row_scale, int* status,
                        cudaStream_t s);
void launch_mx_dequantize(const qlora_mx_tensor* t, void* out, cudaStream_t s);

// Wt[cols, rows] = deq(W)^T, bf16 (the values of qlora_mx_dequantize).
void launch_mx_dequant_t(const qlora_mx_tensor* w, void* Wt, cudaStream_t s);

// out[rows, RP] = RNbf16(in[rows, :r] / row_scale[row]), zero beyond r; no
// division when row_scale is null.  `in` has ldi elements a row; out may be in.
void launch_mx_pad_rows(const void* in, int64_t rows, int r, int ldi, int RP, const float* row_scale,
                        void* out, cudaStream_t s);

// Y[M, N] = deq(x) deq(w)^T + tokad[M, RP] wad[N, RP]^T (bf16 factors, RP a
// multiple of 64 or 0).  With NVFP4 the adapter factors come divided by the
// row scales of x and w.  Returns QLORA_OK or QLORA_ERR_CUDA.
int launch_mx_gemm(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const void* tokad,
                   const void* wad, int RP, void* Y, int* status, cudaStream_t s, int num_sms);

}  // namespace qnf4
