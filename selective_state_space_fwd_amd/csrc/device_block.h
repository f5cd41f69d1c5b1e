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

// The same past L2 (non-temporal): for output that its kernel does not read again, so that the
// inputs' lines stay and the writes drain evenly.
__device__ __forceinline__ void store16_stream(void* p, uint4 v) {
  typedef uint32_t word4 __attribute__((ext_vector_type(4), aligned(2)));
  const word4 q = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(q, static_cast<word4*>(p));
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

// The n (< C) values from p on, the rest zero (nothing past n is read). What lies past n takes
// the last value's address instead of a branch, so that the loads are one trip to memory and not
// one each.
template <typename Elem, int C>
__device__ __forceinline__ void load_part_of(const Elem* p, int n, float (&v)[C]) {
  Elem e[C];
#pragma unroll
  for (int i = 0; i < C; ++i) e[i] = Elem(0);
  if (n > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) e[i] = p[i < n ? i : n - 1];
  }
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = i < n ? widen<Elem>(e[i]) : 0.0f;
}

// v[i] = p[i] for i < n, 0 past it (nothing past it is read). S a multiple of the word.
template <typename Elem, int S>
__device__ __forceinline__ void load_run(const Elem* p, int n, float (&v)[S]) {
  constexpr int N = Vec<Elem>::kN;
  if (n >= S) {
#pragma unroll
    for (int q = 0; q < S / N; ++q) widen_raw16<Elem>(load16_any(p + q * N), v + q * N);
  } else {
    load_part_of<Elem, S>(p, n, v);
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

template <typename Elem, int S>
__device__ __forceinline__ void store_run_stream(Elem* p, int n, const float (&v)[S]) {
  constexpr int N = Vec<Elem>::kN;
  if (n >= S) {
#pragma unroll
    for (int q = 0; q < S / N; ++q) store16_stream(p + q * N, narrow_raw16<Elem>(v + q * N));
  } else {
    store_run<Elem, S>(p, n, v);
  }
}

// N dwords at element alignment.
template <int N>
struct __attribute__((packed, aligned(2))) Dwords {
  uint32_t w[N];
};

// Past L2, as store16_stream.
__device__ __forceinline__ void store_stream(void* p, const Dwords<4>& d) {
  store16_stream(p, make_uint4(d.w[0], d.w[1], d.w[2], d.w[3]));
}

__device__ __forceinline__ void store_stream(void* p, const Dwords<2>& d) {
  typedef uint32_t Pair __attribute__((ext_vector_type(2), aligned(2)));
  __builtin_nontemporal_store(Pair{d.w[0], d.w[1]}, reinterpret_cast<Pair*>(p));
}

// Value c (a constant after unrolling) of storage dwords, and all of them rounded.
template <typename Elem, int N>
__device__ __forceinline__ float few_elem(const Dwords<N>& d, int c) {
  if constexpr (sizeof(Elem) == 4) return __uint_as_float(d.w[c]);
  return (c & 1) ? bf16_hi(d.w[c / 2]) : bf16_lo(d.w[c / 2]);
}

template <typename Elem, int C>
__device__ __forceinline__ void pack_few(const float (&v)[C], Dwords<C * int(sizeof(Elem)) / 4>& d) {
#pragma unroll
  for (int i = 0; i < C * int(sizeof(Elem)) / 4; ++i) {
    if constexpr (sizeof(Elem) == 4)
      d.w[i] = __float_as_uint(v[i]);
    else
      d.w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  }
}

// The n (of C) values from p on, the rest zero.
template <typename Elem, int C>
__device__ __forceinline__ void load_few(const Elem* p, int n, float (&v)[C]) {
  constexpr int N = C * int(sizeof(Elem)) / 4;
  if (n >= C) {
    const Dwords<N> d = *reinterpret_cast<const Dwords<N>*>(p);
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = few_elem<Elem>(d, i);
  } else {
    load_part_of<Elem, C>(p, n, v);
  }
}

template <typename Elem, int C>
__device__ __forceinline__ void store_few(Elem* p, int n, const float (&v)[C]) {
  constexpr int N = C * int(sizeof(Elem)) / 4;
  if (n >= C) {
    Dwords<N> d;
    pack_few<Elem, C>(v, d);
    *reinterpret_cast<Dwords<N>*>(p) = d;
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n) p[i] = narrow<Elem>(v[i]);
  }
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

// ---------------------------------------------------------------- workgroup order

// The place of this workgroup in an order that gives each of the eight XCDs, to which workgroups
// are dealt in turn, one contiguous run: neighbours then share an L2, and an XCD whose tiles
// would all lie at one offset of rows a power of two long (all in the same few channels of
// its L2) gets tiles of every offset.
__device__ __forceinline__ uint32_t xcd_order(uint32_t id, uint32_t total) {
  const uint32_t per = total / 8;
  return id < per * 8 ? (id % 8) * per + id / 8 : id;
}

// ---------------------------------------------------------------- partial rows

// The sum over rows of part[row][col] for one column per thread of a workgroup of kCols columns by
// kSlices slices of the rows, in a fixed order: a slice's rows in order, eight loads at once,
// then the slices. The result is in the threads of slice 0.
template <int kCols, int kSlices>
__device__ __forceinline__ float sum_rows(const float* part, int64_t rows, int64_t cols, int64_t col,
                                          float (&buf)[kSlices][kCols + 1]) {
  const int col_in = threadIdx.x % kCols, slice = threadIdx.x / kCols;
  float a = 0.0f;
  if (col < cols) {
    int64_t r = slice;
    for (; r + 7 * kSlices < rows; r += 8 * kSlices) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = part[(r + i * kSlices) * cols + col];
#pragma unroll
      for (int i = 0; i < 8; ++i) a += v[i];
    }
    for (; r < rows; r += kSlices) a += part[r * cols + col];
  }
  buf[slice][col_in] = a;
  __syncthreads();
  if (slice == 0)
    for (int s = 1; s < kSlices; ++s) a += buf[s][col_in];
  return a;
}

// ---------------------------------------------------------------- cache slots

// Rows of a single-token call name cache slots; rows naming the same slot are successive
// tokens of it, in row order. Of such rows the first takes all (a workgroup each, so the state
// stays in registers between them): `first` says whether row r is it, `next` is the following
// row of the slot (INT32_MAX: none).
struct SlotOrder {
  bool first;
  int next;
};

// The search over all rows' slots for the R rows from r on (their slots in `slot`, < 0: none),
// shared by the kWaves waves of a workgroup (its threads read each slot once), every one of
// whose threads takes part. buf: LDS; a call may follow another with the other `turn` (0 or
// 1) and no barrier between.
template <int kWaves, int R>
__device__ __forceinline__ void slot_order(const int32_t* slots, int batch, int r, const int (&slot)[R],
                                           int (&buf)[2][kWaves][2], int turn, SlotOrder (&order)[R]) {
  bool before[R];
  int next[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    before[k] = false;
    next[k] = INT32_MAX;
  }
#pragma unroll 4
  for (int i = threadIdx.x; i < batch; i += 64 * kWaves) {
    const int s = slots[i];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      before[k] |= s == slot[k] && i < r + k;
      next[k] = s == slot[k] && i > r + k && i < next[k] ? i : next[k];
    }
  }
  // Almost every search finds nothing, so a wave says in one word whether it found any row of
  // the R slots, and the rows themselves are looked for only then.
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < R; ++k) any |= (__ballot(before[k]) != 0 ? 1u : 0u) << k;
  bool later = false;
#pragma unroll
  for (int k = 0; k < R; ++k) later |= next[k] != INT32_MAX;
  if (__ballot(later) != 0) any |= 1u << 31;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) buf[turn][wave][0] = int(any);
  __syncthreads();
  any = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) any |= uint32_t(buf[turn][w][0]);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    order[k].first = ((any >> k) & 1u) == 0;
    order[k].next = INT32_MAX;
  }
  if (any >> 31) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      for (int m = 32; m > 0; m >>= 1) {
        const int other = __shfl_xor(next[k], m, 64);
        next[k] = other < next[k] ? other : next[k];
      }
      if ((threadIdx.x & 63) == 0) buf[turn][wave][1] = next[k];
      __syncthreads();
      for (int w = 0; w < kWaves; ++w)
        order[k].next = buf[turn][w][1] < order[k].next ? buf[turn][w][1] : order[k].next;
      order[k].next = __builtin_amdgcn_readfirstlane(order[k].next);
      __syncthreads();
    }
  }
}

}  // namespace ssm
