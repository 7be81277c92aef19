// page_scale.cuh -- what the stores into pages of one FP8 scale share: the scale that a page's
// largest value needs, held codes under a new scale, and the length of a run of tokens.
#pragma once

#include "kvq_device.cuh"

namespace kvq {

namespace {

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 * 2^8).
__device__ __forceinline__ float page_scale_need(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < 1 ? 1 : e;  // also for a subnormal amax
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// Four E4M3 codes times f (a power of two unless the stored scale was not one).
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h2;
    const uint16_t two = static_cast<uint16_t>((w >> (16 * i)) & 0xFFFFu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    float lo, hi;
    f16x2_to_f32(h2, lo, hi);
    r |= e4m3x2_from_f32(__fmul_rn(lo, f), __fmul_rn(hi, f)) << (16 * i);
  }
  return r | (w & 0x80808080u);  // a NaN code (a row never written) keeps its sign too
}

__device__ __forceinline__ int run_bits(uint32_t m) { return m == 0xFFFFFFFFu ? 32 : __ffs(~m) - 1; }

}  // namespace

}  // namespace kvq
