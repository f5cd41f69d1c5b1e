// Device helpers shared by the kernels around the scan (short convolution, state step, gated
// norm): 16-byte accesses at element alignment, widening and rounding of short runs of
// storage elements, the row order of steps that share a cache slot.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "device_scan.h"

namespace ssm {

// A 16-byte access that needs element alignment only: gfx950 takes dword and larger global
// accesses at any byte address (rows of an odd length, slices of a projection's output), at
// the cost of at most one more cache line per access.
struct __attribute__((packed, aligned(2))) Any16 {
  uint32_t w[4];
};

__device__ __forceinline__ uint4 load16_any(const void* p) {
  const Any16 r = *static_cast<const Any16*>(p);
  return make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
}

__device__ __forceinline__ void store16_any(void* p, uint4 v) {
  Any16 r;
  r.w[0] = v.x;
  r.w[1] = v.y;
  r.w[2] = v.z;
  r.w[3] = v.w;
  *static_cast<Any16*>(p) = r;
}

template <typename Elem>
__device__ __forceinline__ float widen(Elem v);
template <>
__device__ __forceinline__ float widen<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float widen<uint16_t>(uint16_t v) {
  return bf16_lo(v);
}

// Rounded to nearest-even (bf16) or kept (fp32).
template <typename Elem>
__device__ __forceinline__ Elem narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float v) {
  return uint16_t(pack_bf16x2(v, 0.0f));
}

// The 16-byte word of Vec<Elem>::kN values.
template <typename Elem>
__device__ __forceinline__ uint4 narrow_raw16(const float* v);
template <>
__device__ __forceinline__ uint4 narrow_raw16<float>(const float* v) {
  return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                    __float_as_uint(v[3]));
}
template <>
__device__ __forceinline__ uint4 narrow_raw16<uint16_t>(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// v[i] = p[i] for i < n, 0 past it (nothing past it is read). S a multiple of the word.
template <typename Elem, int S>
__device__ __forceinline__ void load_run(const Elem* p, int n, float (&v)[S]) {
  constexpr int N = Vec<Elem>::kN;
  if (n >= S) {
#pragma unroll
    for (int q = 0; q < S / N; ++q) widen_raw16<Elem>(load16_any(p + q * N), v + q * N);
  } else {
#pragma unroll
    for (int i = 0; i < S; ++i) v[i] = i < n ? widen<Elem>(p[i]) : 0.0f;
  }
}

// p[i] = v[i] for i < n.
template <typename Elem, int S>
__device__ __forceinline__ void store_run(Elem* p, int n, const float (&v)[S]) {
  constexpr int N = Vec<Elem>::kN;
  if (n >= S) {
#pragma unroll
    for (int q = 0; q < S / N; ++q) store16_any(p + q * N, narrow_raw16<Elem>(v + q * N));
  } else {
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (i < n) p[i] = narrow<Elem>(v[i]);
  }
}

// The storage word of n <= kN elements, zeros past them.
template <typename Elem>
__device__ __forceinline__ uint4 load_word_n(const Elem* p, int n) {
  constexpr int N = Vec<Elem>::kN;
  if (n >= N) return load16_any(p);
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = i < n ? widen<Elem>(p[i]) : 0.0f;
  return narrow_raw16<Elem>(v);
}

// Element c (a constant after unrolling) of a storage word, widened.
template <typename Elem>
__device__ __forceinline__ float word_elem(const uint4& w, int c);
template <>
__device__ __forceinline__ float word_elem<float>(const uint4& w, int c) {
  return __uint_as_float(c == 0 ? w.x : c == 1 ? w.y : c == 2 ? w.z : w.w);
}
template <>
__device__ __forceinline__ float word_elem<uint16_t>(const uint4& w, int c) {
  const uint32_t d = c < 2 ? w.x : c < 4 ? w.y : c < 6 ? w.z : w.w;
  return (c & 1) ? bf16_hi(d) : bf16_lo(d);
}

// silu(p) = p sigmoid(p), and its derivative sigmoid(p) (1 + p (1 - sigmoid(p))).
__device__ __forceinline__ float sigmoid_f(float p) {
  return rcp_hw(1.0f + exp2_hw(-p * kLog2e));
}
__device__ __forceinline__ float silu_f(float p) { return p * sigmoid_f(p); }
__device__ __forceinline__ float silu_grad_f(float p) {
  const float s = sigmoid_f(p);
  return s * __builtin_fmaf(p, 1.0f - s, 1.0f);
}

// ---------------------------------------------------------------- sums over lanes

template <int kCtrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, true));
}

// The sum over each aligned group of 2^LG lanes, in every lane of it, in a fixed order: pairs
// and quads by quad_perm; rows of 8 and 16 by the mirrors (every lane of a half holds the
// half's sum by then); rows of 16 across a wave through the LDS crossbar.
template <int LG>
__device__ __forceinline__ float sum_lanes(float v) {
  if constexpr (LG >= 1) v = dpp_add<0xB1>(v);   // quad_perm 1,0,3,2
  if constexpr (LG >= 2) v = dpp_add<0x4E>(v);   // quad_perm 2,3,0,1
  if constexpr (LG >= 3) v = dpp_add<0x141>(v);  // row_half_mirror
  if constexpr (LG >= 4) v = dpp_add<0x140>(v);  // row_mirror
  if constexpr (LG >= 5) v += __shfl_xor(v, 16, 64);
  if constexpr (LG >= 6) v += __shfl_xor(v, 32, 64);
  return v;
}

// ---------------------------------------------------------------- cache slots

// Rows of a single-token call name cache slots; rows naming the same slot are successive
// tokens of it, in row order. Of such rows the first takes all (a workgroup each, so the state
// stays in registers between them): `first` says whether row r is it, `next` is the following
// row of the slot (INT32_MAX: none). Every lane of the wave takes part.
struct SlotOrder {
  bool first;
  int next;
};

__device__ __forceinline__ SlotOrder slot_order(const int32_t* slots, int batch, int r, int slot) {
  bool before = false;
  int next = INT32_MAX;
#pragma unroll 4
  for (int i = threadIdx.x & 63; i < batch; i += 64) {
    const bool same = slots[i] == slot;
    before |= same && i < r;
    next = same && i > r && i < next ? i : next;
  }
  SlotOrder o;
  o.first = __ballot(before) == 0;
  if (__ballot(next != INT32_MAX) != 0) {
    for (int m = 32; m > 0; m >>= 1) {
      const int other = __shfl_xor(next, m, 64);
      next = other < next ? other : next;
    }
  }
  o.next = __builtin_amdgcn_readfirstlane(next);
  return o;
}

}  // namespace ssm
