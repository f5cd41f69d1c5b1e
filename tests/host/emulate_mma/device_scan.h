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
// A buffer whose accesses at or past its length read 0 and are dropped.
struct Buf {
  char* p;
  uint32_t bytes;
  Buf(const void* base, uint32_t n) : p(static_cast<char*>(const_cast<void*>(base))), bytes(n) {}
  template <typename T>
  T load(uint32_t off, uint32_t soff = 0) const {
    T v{};
    if (off < bytes) memcpy(&v, p + off + soff, sizeof(T));
    return v;
  }
  template <typename T>
  void store(T v, uint32_t off) const {
    if (off < bytes) memcpy(p + off, &v, sizeof(T));
  }
  uint4 load16(uint32_t off, uint32_t soff = 0) const { return load<uint4>(off, soff); }
  uint32_t load4(uint32_t off) const { return load<uint32_t>(off); }
  uint32_t load2(uint32_t off) const { return load<uint16_t>(off); }
  void store16(uint4 v, uint32_t off) const { store(v, off); }
  void store8(uint2 v, uint32_t off) const { store(v, off); }
  void store4(uint32_t v, uint32_t off) const { store(v, off); }
  void store2(uint16_t v, uint32_t off) const { store(v, off); }
};
}  // namespace ssm
