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

// A launch that may begin when every CTA of the kernel before it has called
// grid_launch_dependents or ended.
template <typename... P, typename... A>
void launch_dependent(void (*kern)(P...), dim3 grid, dim3 block, bool dependent, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// beside (here and below): launched beside the kernel before it, of which it reads
// nothing, and ending after it.
void launch_mx_quantize(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ld, int format,
                        uint8_t* packed, uint8_t* scales, float* row_scale, bool beside, int* status,
                        cudaStream_t s);
struct Dropout;
// dX [M, K] (bf16, in place) += D c (sU [M, RP] At [K, RP]^T), K % 64 == 0.
// It reads nothing before the kernel before it has ended.
void launch_mx_rank_add(const void* sU, const void* At, int RP, int M, int K, void* dX, const Dropout& drop,
                        cudaStream_t s);

// Few tokens (M <= kMxPrepTokens): X [M, K] bf16 quantised (scales of rows past M
// are left as they are) and, with r > 0 and T = X A^T, sT [M, r] = RNbf16(s T)
// and T_save = RNbf16(T) (may be null).  K <= kMxPrepMaxK.
constexpr int kMxPrepTokens = 64;
constexpr int kMxPrepMaxK = 3 * 256 * 32;
void launch_mx_prep(const void* X, int M, int K, const void* A, int r, int format, uint8_t* packed, uint8_t* scales,
                    float* row_scale, float s, void* sT, void* T_save, int* status, cudaStream_t st);

void launch_mx_dequantize(const qlora_mx_tensor* t, void* out, cudaStream_t s);

// Wt[cols, rows] = deq(W)^T, bf16 (the values of qlora_mx_dequantize).
void launch_mx_dequant_t(const qlora_mx_tensor* w, void* Wt, bool beside, cudaStream_t s);

// out[rows, RP] = RNbf16(in[rows, :r] / row_scale[row]), zero beyond r; no
// division when row_scale is null.  `in` has ldi elements a row; out may be in.
void launch_mx_pad_rows(const void* in, int64_t rows, int r, int ldi, int RP, const float* row_scale,
                        void* out, cudaStream_t s);

// The adapter term of a product: none (RP = r = 0), bf16 factors of RP columns
// (a multiple of 64) as extra K steps, tok [M, RP] and wt [N, RP] (with NVFP4
// divided by the row scales of x and w), or, where mx_adapter_in_epilogue, sT
// [M, r] and B [N, r] as they are, added by the epilogue.
struct MxAdapter {
  int RP = 0;
  const void* tok = nullptr;
  const void* wt = nullptr;
  int r = 0;
  const void* sT = nullptr;
  const void* B = nullptr;
};

// Whether the product of these sizes adds the adapter in its epilogue: with few
// tokens, and where the paired kernel has one round of tiles (a longer one
// would wait for its epilogues; one round saves the launch that prepares B).
bool mx_adapter_in_epilogue(int M, int N, int K, int num_sms);

// Y[M, N] = deq(x) deq(w)^T + the adapter's term.  after_prep: launched as the
// dependent of the kernel before it (launch_mx_prep, launch_mx_quantize or
// launch_mx_down), with whose end x, sT, tok and wt are complete: the kernel that
// writes wt (launch_mx_pad_rows) may still run when this one starts.  Only w, its
// scales and B may be read before the wait for that end.  QLORA_OK or QLORA_ERR_CUDA.
int launch_mx_gemm(const qlora_mx_tensor* x, const qlora_mx_tensor* w, const MxAdapter& ad, bool after_prep, void* Y,
                   int* status, cudaStream_t s, int num_sms);

// With S = Z R^T, Z [M, L] and R [r, L] (r_rows: R^T [L, r]) bf16: pad [M, RP] = RNbf16(s S /
// row_scale[m]), zero beyond r (row_scale null: no division), and out [M, r] =
// RNbf16(S); either may be null.  L % 8 == 0.  after: kBeside, launched beside the
// kernel before it (launch_mx_quantize), which wrote row_scale and nothing else
// that is read here; kWaits, only the set-up is beside it.  QLORA_OK or
// QLORA_ERR_CUDA.
enum class After { kEnds, kBeside, kWaits };
int launch_mx_down(const void* Z, const void* R, bool r_rows, int M, int L, int r, int RP, float s,
                   const float* row_scale, void* pad, void* out, After after, int* status, cudaStream_t st, int num_sms);

// dA [r, K] = RNbf16(sU^T Xd), dB [N, r] = RNbf16(s dY^T T) over M tokens; sU has
// ldu columns.  Only its set-up is beside the kernel before it.  QLORA_OK or
// QLORA_ERR_CUDA.
int launch_mx_outer(const void* Xd, int K, const void* sU, int ldu, void* dA, const void* dY, int N, const void* T,
                    float s, void* dB, int M, int r, int* status, cudaStream_t st, int num_sms);

// At [K, RP] = A [r, K]^T, zero beyond r.
void launch_mx_transpose(const void* A, int r, int K, int RP, void* At, cudaStream_t s);

// dX [M, K] = dY deq(W) + sU A over RP = 64 na columns of sU [M, RP] (na = 0: the
// first term alone), W expanded inside the product; mx_dx_expands_inside: whether
// that is the faster way for these sizes.  beside: launched as the dependent of the
// kernel before it, of whose results it reads sU alone.  QLORA_OK or QLORA_ERR_CUDA.
bool mx_dx_expands_inside(int M, int N, int K, int na, int num_sms);
int launch_mx_dx(const qlora_mx_tensor* w, const void* dY, int M, const void* A, int r, const void* sU, int RP, int na,
                 void* dX, bool beside, int* status, cudaStream_t s, int num_sms);

}  // namespace qnf4
