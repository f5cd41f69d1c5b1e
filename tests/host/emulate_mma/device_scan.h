// The helpers of csrc/device_scan.h that the linear-attention kernels use, for a CPU build.
#pragma once
#include "device_math.h"

namespace ssm {
template <typename Elem>
struct Vec {
  static constexpr int kN = 16 / int(sizeof(Elem));
};
template <typename Elem>
inline void widen_raw16(uint4 w, float* v) {
  const uint32_t d[4] = {w.x, w.y, w.z, w.w};
  for (int i = 0; i < Vec<Elem>::kN; ++i)
    v[i] = sizeof(Elem) == 4 ? __uint_as_float(d[i % 4]) : i % 2 ? bf16_hi(d[i / 2]) : bf16_lo(d[i / 2]);
}
}  // namespace ssm
