// The dropout mask's generator for kernels that apply it themselves.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace qnf4 {

// A Philox block's keep bits, as dropout_keep8 (common.cuh) draws them, with fewer
// instructions.
// What is left, 18 products of 64 x 64 bits a block, is bound by the integer
// multiplier: 40 us for the 3.7 M blocks of a 8192 x 3584 tensor, of the 50 us
// that bf16 dropout of it takes (fp32 8192 x 8192: 103 us, 5.2 TB/s).
//  * the keys of the ten rounds are the same for every thread: they come as
//    kernel arguments (constant operands);
//  * key word 1 and counter words 1 to 3 start at 0, so round 1 has one product
//    and in round 2 the other one has only constant factors;
//  * a 24-bit uniform u >= thr is compared as a 32-bit word >= thr << 8 whose
//    top 24 bits are u (thr < 2^24 as p < 1).
struct DropoutKeys {
  uint64_t k0[10];         // seed + r * W0
  uint64_t h, l;           // the constant product of round 2: M0 * k0[0]
  uint32_t thr8;           // thr << 8 (0 keeps everything)
  float scale;
};

constexpr uint64_t kM0 = 0xD2E7470EE14C6C93ull, kM1 = 0xCA5A826395121157ull, kW1 = 0xBB67AE8584CAA73Bull;

__device__ __forceinline__ void mul128(uint64_t a, uint64_t m, uint64_t& hi, uint64_t& lo) {
  const unsigned __int128 p = (unsigned __int128)a * m;
  hi = (uint64_t)(p >> 64);
  lo = (uint64_t)p;
}

struct Draw {
  uint64_t w[4];
  __device__ __forceinline__ bool keep(int i, uint32_t thr8) const {
    const uint32_t hi = (uint32_t)(w[i >> 1] >> 32), lo = (uint32_t)w[i >> 1];
    return ((i & 1) ? __funnelshift_l(lo, hi, 24) : hi) >= thr8;
  }
};

__device__ __forceinline__ Draw draw8(uint64_t blk, const DropoutKeys& k) {
  uint64_t h0, l0, h1, l1, c0, c1, c2, c3;
  mul128(blk, kM0, h0, l0);                        // round 1: (blk, 0, 0, 0)
  c2 = h0;                                         // c0 = k0[0], c1 = 0, c3 = l0
  c3 = l0;
  mul128(c2, kM1, h1, l1);                         // round 2
  c0 = h1 ^ k.k0[1];
  c1 = l1;
  c2 = k.h ^ c3 ^ kW1;
  c3 = k.l;
#pragma unroll
  for (int r = 2; r < 10; ++r) {
    mul128(c0, kM0, h0, l0);
    mul128(c2, kM1, h1, l1);
    c0 = h1 ^ c1 ^ k.k0[r];
    c1 = l1;
    c2 = h0 ^ c3 ^ (kW1 * (uint64_t)r);
    c3 = l0;
  }
  return Draw{{c0, c1, c2, c3}};
}

inline DropoutKeys make_keys(const Dropout& d) {
  DropoutKeys k{};
  for (int r = 0; r < 10; ++r) k.k0[r] = d.seed + (uint64_t)r * 0x9E3779B97F4A7C15ull;
  const unsigned __int128 p = (unsigned __int128)kM0 * k.k0[0];
  k.h = (uint64_t)(p >> 64);
  k.l = (uint64_t)p;
  k.thr8 = d.thr << 8;
  k.scale = d.scale;
  return k;
}

}  // namespace qnf4
