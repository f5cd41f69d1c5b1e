// The arithmetic of csrc/device_math.h that the kernels around the scan use, for a CPU build.
#pragma once
#include <hip/hip_runtime.h>

namespace ssm {
constexpr float kLog2e = 1.44269504088896340736f;
inline float exp2_hw(float x) { return exp2f(x); }
inline float rcp_hw(float x) { return 1.0f / x; }
inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
inline uint32_t bf16_bits(float v) {  // to nearest-even
  const uint32_t u = __float_as_uint(v);
  if (v != v) return (u >> 16) | 0x40u;
  return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
}
inline uint32_t pack_bf16x2(float lo, float hi) { return bf16_bits(lo) | bf16_bits(hi) << 16; }
}  // namespace ssm
