// Values of microscaled 4-bit elements.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "mx.h"

namespace qnf4 {

// Eight E2M1 codes -> four f16x2 words (exact).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t c, uint32_t* h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}

__device__ __forceinline__ float from_e4m3(uint32_t b) {
  uint32_t h;
  const uint16_t p = (uint16_t)b;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(p));
  return f16x2_to_f32(h).x;
}
// 2^(b - 127); byte 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ float from_e8m0(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255u ? 0x7FFFFFFFu : b << 23);
}

template <int FMT>
__device__ __forceinline__ float mx_scale_value(uint32_t b) {
  return FMT == QLORA_NVFP4 ? from_e4m3(b) : from_e8m0(b);
}

// Eight elements as bf16: RNbf16(RN32(q S rs)); q S is exact.
template <int FMT>
__device__ __forceinline__ uint4 mx_values8(uint32_t c, float S, float rs) {
  uint32_t h[4], o[4];
  e2m1x8_to_f16(c, h);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = f16x2_to_f32(h[j]);
    float a = __fmul_rn(f.x, S), b = __fmul_rn(f.y, S);
    if (FMT == QLORA_NVFP4) { a = __fmul_rn(a, rs); b = __fmul_rn(b, rs); }
    o[j] = pack_bf16x2(a, b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace qnf4
