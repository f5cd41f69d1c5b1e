// Device helpers of the linear-attention kernels: tiles of head rows staged in LDS, operands of the
// matrix instructions read from them along rows or columns, fp32 values as bf16 pieces, and the
// running decays of a chunk of steps.
//
// Operand layout (v_mfma_f32_16x16x32_bf16): lane l, r = l % 16, g = l / 16, holds the contraction
// values 8g..8g+7 of row r of the first operand, and of column r of the second; the result
// has rows 4g..4g+3 of column r. A fragment is the same for both sides, so swapping the two
// transposes the result. fp32 storage takes v_mfma_f32_16x16x4_f32 eight times on the same
// fragments: its lane group g supplies contraction value g, here value 8g + i of the i-th.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_block.h"
#include "linattn_launch.h"

namespace ssm {

typedef __bf16 la_bf16x8 __attribute__((ext_vector_type(8)));
typedef float la_f32x4 __attribute__((ext_vector_type(4)));
typedef short la_s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) la_s16x4 la_lds_s16x4;

constexpr int kLaThreads = 256;

template <typename Elem>
constexpr int chunk_of() {
  return linattn_chunk(sizeof(Elem) == 2 ? Io::BF16 : Io::F32);
}

// A barrier for LDS only: loads on their way from memory and results on their way out go on
// across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Eight contraction values of one row (or column).
template <typename Elem>
struct Frag;
template <>
struct Frag<uint16_t> {
  uint4 w;
};
template <>
struct Frag<float> {
  float v[8];
};

__device__ __forceinline__ la_f32x4 mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, la_f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(la_bf16x8, a.w),
                                                 __builtin_bit_cast(la_bf16x8, b.w), c, 0, 0, 0);
}
__device__ __forceinline__ la_f32x4 mma(const Frag<float>& a, const Frag<float>& b, la_f32x4 c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

// Eight fp32 values as an operand next to storage type Elem: N bf16 pieces, each the rounding of
// what the ones before leave (8 bits of the significand each, so three hold all 24), or the
// values themselves in fp32. What an infinity leaves is NaN, so that an infinite state or value (above bf16's
// largest, 3.39e38, too) gives NaN where fp32 storage may give an infinity: a number in that place would be
// a v_max_f32 more for each value, 1 to 3% of the calls (b8, 32 heads of 128 x 64: 109.2 us, 112.8 with it).
template <typename Elem, int N>
struct Pieces;
template <int N>
struct Pieces<uint16_t, N> {
  static constexpr int kCount = N;
  Frag<uint16_t> f[N];
  __device__ __forceinline__ void split(const float (&x)[8]) {
    float rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rest[i] = x[i];
#pragma unroll
    for (int p = 0; p < N; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = pack_bf16x2(rest[2 * i], rest[2 * i + 1]);
        rest[2 * i] -= bf16_lo(w[i]);
        rest[2 * i + 1] -= bf16_hi(w[i]);
      }
      f[p].w = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};
template <int N>
struct Pieces<float, N> {
  static constexpr int kCount = 1;
  Frag<float> f;
  __device__ __forceinline__ void split(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = x[i];
  }
};

// Piece p of kCount.
template <int N>
__device__ __forceinline__ const Frag<uint16_t>& piece(const Pieces<uint16_t, N>& a, int p) {
  return a.f[p];
}
template <int N>
__device__ __forceinline__ const Frag<float>& piece(const Pieces<float, N>& a, int) {
  return a.f;
}

__device__ __forceinline__ void widen_frag(const Frag<uint16_t>& f, float (&v)[8]) {
  widen_raw16<uint16_t>(f.w, v);
}
__device__ __forceinline__ void widen_frag(const Frag<float>& f, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = f.v[i];
}

// Elements between rows of a staged tile of D columns: a little more than the row, so that the 16
// rows of an operand read start in different banks.
template <typename Elem>
__host__ __device__ constexpr int la_pitch(int D) {
  return D + 16 / int(sizeof(Elem));
}

// Contraction values k0 + 8g .. + 7 of row `row`.
__device__ __forceinline__ Frag<uint16_t> row_frag(const uint16_t* tile, int pitch, int row, int k0) {
  const int g = (threadIdx.x & 63) >> 4;
  Frag<uint16_t> f;
  f.w = *reinterpret_cast<const uint4*>(tile + row * pitch + k0 + 8 * g);
  return f;
}
__device__ __forceinline__ Frag<float> row_frag(const float* tile, int pitch, int row, int k0) {
  const int g = (threadIdx.x & 63) >> 4;
  const float4 a = *reinterpret_cast<const float4*>(tile + row * pitch + k0 + 8 * g);
  const float4 b = *reinterpret_cast<const float4*>(tile + row * pitch + k0 + 8 * g + 4);
  return Frag<float>{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// Column c0 + r, contraction over rows: values of rows s0 + 8g .. + 7. bf16 through the transposing
// LDS read: of each 16 lanes, lane i supplies the address of four columns (4 (i % 4) on) of
// row i / 4 and receives column i of the four rows.
__device__ __forceinline__ Frag<uint16_t> transposed(const uint16_t* p, int pitch) {
  const la_s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((la_lds_s16x4*)p);
  const la_s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((la_lds_s16x4*)(p + 4 * pitch));
  const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
  return Frag<uint16_t>{make_uint4(x.x, x.y, y.x, y.y)};
}
__device__ __forceinline__ Frag<float> transposed(const float* p, int pitch) {
  Frag<float> f;
#pragma unroll
  for (int i = 0; i < 8; ++i) f.v[i] = p[i * pitch];
  return f;
}
__device__ __forceinline__ Frag<uint16_t> col_frag(const uint16_t* tile, int pitch, int s0, int c0) {
  const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
  return transposed(tile + (s0 + 8 * g + (r >> 2)) * pitch + c0 + 4 * (r & 3), pitch);
}
__device__ __forceinline__ Frag<float> col_frag(const float* tile, int pitch, int s0, int c0) {
  const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
  return transposed(tile + (s0 + 8 * g) * pitch + c0 + r, pitch);
}

// Half `odd` of 32 columns from c0 on, such that the results' rows 4g .. 4g + 3 of the two halves are
// columns c0 + 8g .. + 3 and c0 + 8g + 4 .. + 7: a state kept as results then is, pair by pair, the
// operand of its eight contraction values as it stands.
__device__ __forceinline__ Frag<uint16_t> col_frag_paired(const uint16_t* tile, int pitch, int s0, int c0, int odd) {
  const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
  return transposed(tile + (s0 + 8 * g + (r >> 2)) * pitch + c0 + 8 * (r & 3) + 4 * odd, pitch);
}
__device__ __forceinline__ Frag<float> col_frag_paired(const float* tile, int pitch, int s0, int c0, int odd) {
  const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
  return transposed(tile + (s0 + 8 * g) * pitch + c0 + 8 * (r >> 2) + (r & 3) + 4 * odd, pitch);
}

// Four values of a result (rows 4g .. 4g + 3 of a column) as a run of four storage elements in LDS.
__device__ __forceinline__ void put4(uint16_t* p, const la_f32x4& v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void put4(float* p, const la_f32x4& v) { *reinterpret_cast<la_f32x4*>(p) = v; }

// Four storage elements of LDS.
__device__ __forceinline__ la_f32x4 get4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return la_f32x4{bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
}
__device__ __forceinline__ la_f32x4 get4(const float* p) { return *reinterpret_cast<const la_f32x4*>(p); }

// Whether any value of the operands given is infinite or NaN: a pair of steps that a chunk's product leaves out
// by a weight of 0 would put 0 x infinity, NaN, into results that the value has no part in. Of every value the exponent
// alone, plus one, carries into the sign's place where it is all ones.
struct NotFinite {
  uint32_t seen = 0, signs = 0;
  __device__ __forceinline__ void add(const Frag<uint16_t>& f) {
    for (uint32_t w : {f.w.x, f.w.y, f.w.z, f.w.w}) seen |= (w & 0x7f807f80u) + 0x00800080u;
    signs = 0x80008000u;
  }
  __device__ __forceinline__ void add(const Frag<float>& f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) seen |= (__float_as_uint(f.v[i]) & 0x7f800000u) + 0x00800000u;
    signs = 0x80000000u;
  }
  // In any lane of the wave.
  __device__ __forceinline__ bool any() const { return __ballot((seen & signs) != 0) != 0; }
};

// x, such that nothing formed of it is formed ahead of a loop around it (where it would hold registers).
__device__ __forceinline__ int not_ahead(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ float widen_one(uint16_t v) { return bf16_lo(v); }
__device__ __forceinline__ float widen_one(float v) { return v; }

// acc += the sum over steps [from, to) of weight (at w + step * w_step) times four values (at x + step * x_step), those
// steps alone: what a product over whole blocks of steps gives where every value is finite.
template <typename Elem>
__device__ __forceinline__ la_f32x4 steps_alone(const Elem* w, int w_step, const Elem* x, int x_step, int from, int to,
                                                la_f32x4 acc) {
#pragma unroll 1
  for (int s = from; s < to; ++s) {
    const float weight = widen_one(w[s * w_step]);
    const la_f32x4 v = get4(x + s * x_step);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(weight, v[e], acc[e]);
  }
  return acc;
}

// A byte offset past every buffer: loads there read 0, stores are dropped. Loads and stores go
// through buffer resources with it in the place of a branch, so that nothing but their use waits.
constexpr uint32_t kLaOob = 0x80000000u;
constexpr uint32_t kLaBytes = 0x7fffffffu;  // offsets in use are below it (linattn_reach)

// A tile of C steps x D columns on its way from memory to LDS, spread over the workgroup's threads.
// kWhole: rows of whole 16-byte words at 4-byte aligned addresses, a load a word; else a load an
// element.
template <typename Elem, int C, int D, bool kWhole, int kThreads = kLaThreads>
struct TileLoad {
  static constexpr int kN = Vec<Elem>::kN, kRow = D / kN, kWords = C * kRow / kThreads;
  static constexpr int kStep = kThreads / kRow;  // rows from one of a thread's words to the next
  static_assert(C * kRow % kThreads == 0 && kThreads % kRow == 0, "whole words, whole rows");
  uint4 w[kWords];

  // Rows [0, rows) of `dim` elements, `step` bytes apart; zeros elsewhere (nothing there is read).
  __device__ __forceinline__ void load(const Elem* base, uint32_t step, int rows, int dim) {
    constexpr uint32_t E = sizeof(Elem);
    const Buf b(base, kLaBytes);
    const int row = int(threadIdx.x) / kRow, col = (int(threadIdx.x) % kRow) * kN;
    const uint32_t off = uint32_t(row) * step + uint32_t(col) * E;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const bool on = row < rows - i * kStep;
      const uint32_t s = uint32_t(i * kStep) * step;
      if constexpr (kWhole) {
        w[i] = b.load16(on && col < dim ? off : kLaOob, s);
      } else if constexpr (E == 4) {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = b.load4(on && col + e < dim ? off + s + 4 * e : kLaOob);
        w[i] = make_uint4(x[0], x[1], x[2], x[3]);
      } else {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = b.load2(on && col + 2 * e < dim ? off + s + 4 * e : kLaOob) |
                 b.load2(on && col + 2 * e + 1 < dim ? off + s + 4 * e + 2 : kLaOob) << 16;
        w[i] = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  }
  __device__ __forceinline__ void store(Elem* tile) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const int at = int(threadIdx.x) + i * kThreads, row = at / kRow, col = (at % kRow) * kN;
      *reinterpret_cast<uint4*>(tile + row * la_pitch<Elem>(D) + col) = w[i];
    }
  }
};

// Four neighbouring elements at byte offset off, of which the first n are stored (none where !on).
template <typename Elem, bool kWhole>
__device__ __forceinline__ void store4_at(const Buf& b, uint32_t off, int n, bool on, const la_f32x4& v) {
  if constexpr (sizeof(Elem) == 4) {
    if constexpr (kWhole) {
      b.store16(make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])),
                on && n > 0 ? off : kLaOob);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) b.store4(__float_as_uint(v[e]), on && e < n ? off + 4 * e : kLaOob);
    }
  } else {
    const uint2 w = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    if constexpr (kWhole) {
      b.store8(w, on && n > 0 ? off : kLaOob);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        b.store2(uint16_t((e < 2 ? w.x : w.y) >> (16 * (e & 1))), on && e < n ? off + 2 * e : kLaOob);
    }
  }
}

// ---------------------------------------------------------------- decays

__device__ __forceinline__ double dpp_f64(double v, int lane_of) {
  const int2 w = __builtin_bit_cast(int2, v);
  int2 o;
  o.x = __builtin_amdgcn_readlane(w.x, lane_of);
  o.y = __builtin_amdgcn_readlane(w.y, lane_of);
  return __builtin_bit_cast(double, o);
}
template <int kCtrl>
__device__ __forceinline__ double dpp_add_f64(double v) {
  const int2 w = __builtin_bit_cast(int2, v);
  int2 o;
  o.x = __builtin_amdgcn_update_dpp(0, w.x, kCtrl, 0xf, 0xf, true);
  o.y = __builtin_amdgcn_update_dpp(0, w.y, kCtrl, 0xf, 0xf, true);
  return v + __builtin_bit_cast(double, o);
}
// Inclusive sums over the lanes of a wave, in 64 bits.
__device__ __forceinline__ double wave_prefix_f64(double v) {
  v = dpp_add_f64<0x111>(v);  // row_shr 1, 2, 4, 8
  v = dpp_add_f64<0x112>(v);
  v = dpp_add_f64<0x114>(v);
  v = dpp_add_f64<0x118>(v);
  const double a = dpp_f64(v, 15), b = dpp_f64(v, 31), c = dpp_f64(v, 47);
  const int row = int(threadIdx.x & 63) >> 4;
  return v + (row >= 1 ? a : 0.0) + (row >= 2 ? b : 0.0) + (row >= 3 ? c : 0.0);
}

// Sums of floats over some of a wave's lanes. They only add: what a lane does not sum leaves no trace in
// it, however large, infinite or NaN.
template <int kCtrl>
__device__ __forceinline__ float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_value(float v, int lane_of) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane_of));
}
// Over the lanes of a row of 16: up to and with this one, and from it on.
__device__ __forceinline__ float row_prefix(float v) {
  v = dpp_add<0x111>(v);  // row_shr 1, 2, 4, 8
  v = dpp_add<0x112>(v);
  v = dpp_add<0x114>(v);
  return dpp_add<0x118>(v);
}
__device__ __forceinline__ float row_suffix(float v) {
  return dpp_move<0x140>(row_prefix(dpp_move<0x140>(v)));  // row_mirror
}
// Over the lanes of a wave: before this one, and from it on.
__device__ __forceinline__ float wave_before(float v) {
  v = row_prefix(v);
  const float a = lane_value(v, 15), b = lane_value(v, 31), c = lane_value(v, 47);
  const int row = int(threadIdx.x & 63) >> 4;
  return dpp_move<0x111>(v) + (row >= 1 ? a : 0.0f) + (row >= 2 ? b : 0.0f) + (row >= 3 ? c : 0.0f);
}
__device__ __forceinline__ float wave_from(float v) {
  v = row_suffix(v);
  const float a = lane_value(v, 16), b = lane_value(v, 32), c = lane_value(v, 48);
  const int row = int(threadIdx.x & 63) >> 4;
  return v + (row <= 2 ? c : 0.0f) + (row <= 1 ? b : 0.0f) + (row <= 0 ? a : 0.0f);
}
// The log decay of a step in units of log 2. Below -1e4 it is -1e4, whose exponential is zero all
// the same, so that a reset (-inf) leaves finite sums.
__device__ __forceinline__ double log2_decay(float g) {
  const float x = g < -1e4f ? -1e4f : g;
  return double(x) * 1.4426950408889634074;
}

// A chunk's running decays in log 2: the sums in 64 bits kept as two floats each, because the
// decay between two steps is a difference of sums that may be far larger than it.
template <int C>
struct Decays {
  struct Sum {
    float hi, lo;
  };
  Sum sum[C];     // over the steps up to and with t
  float into[C];  // exp of it: from the chunk's start to t
  float onto[C];  // from s to the chunk's end
  float total;    // over the chunk

  // Lane t < C of one wave holds the step's log decay (0 behind the end). Returns the log2 sum.
  __device__ __forceinline__ double set(float step) {
    const int l = threadIdx.x & 63;
    const double cs = wave_prefix_f64(log2_decay(step)), all = dpp_f64(cs, C - 1);
    if (l < C) {
      const float h = float(cs);
      sum[l] = Sum{h, float(cs - double(h))};
      into[l] = exp2_hw(h);
      onto[l] = exp2_hw(float(all - cs));
      if (l == 0) total = exp2_hw(float(all));
    }
    return all;
  }
  // As set, for the gradient, where a NaN or infinite decay must not be between steps that both lie behind it (in the
  // forward, and in the states, it is in all that is behind it anyway): it is kept out of the sums, and is NaN in
  // `into`, `onto` and `total`, of which each result that such a decay is in has one.
  __device__ __forceinline__ void set_apart(float step) {
    if (__builtin_expect(set(step) < 1e30, 1)) return;
    const int l = threadIdx.x & 63;
    const bool counts = step <= 1e4f;
    const unsigned long long odd = __ballot(!counts), from = odd & ((2ull << l) - 1), behind = odd >> l >> 1;
    const double cs = wave_prefix_f64(counts ? log2_decay(step) : 0.0), all = dpp_f64(cs, C - 1);
    const float nan = __builtin_nanf("");
    if (l < C) {
      const float h = float(cs);
      sum[l] = Sum{h, float(cs - double(h))};
      into[l] = from ? nan : exp2_hw(h);
      onto[l] = behind ? nan : exp2_hw(float(all - cs));
      if (l == 0) total = nan;
    }
  }
  // From s0 + e to t, e < 4. All four whatever comes of them: a condition around one would put its
  // loads and exponential in a branch of their own.
  __device__ __forceinline__ void between(int t, int s0, float (&keep)[4]) const {
    const Sum to = sum[t];
    Sum from[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) from[e] = sum[s0 + e];
#pragma unroll
    for (int e = 0; e < 4; ++e) keep[e] = exp2_hw((to.hi - from[e].hi) + (to.lo - from[e].lo));
  }
  // From s to t0 + e.
  __device__ __forceinline__ void onwards(int s, int t0, float (&keep)[4]) const {
    const Sum from = sum[s];
    Sum to[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e] = sum[t0 + e];
#pragma unroll
    for (int e = 0; e < 4; ++e) keep[e] = exp2_hw((to[e].hi - from.hi) + (to[e].lo - from.lo));
  }
};

// The log decay of step t0 + lane, 0 at and past `rows` and without g (nothing there is read). A load
// without a branch, by every wave: a later wait for an older load can then leave it in flight.
__device__ __forceinline__ float load_decay(const float* g, int64_t step, int64_t t0, int rows, int64_t from = 0) {
  const int l = threadIdx.x & 63;
  const Buf b(g + t0 * step + from, kLaBytes);
  return __uint_as_float(b.load4(g && l < rows ? uint32_t(l) * uint32_t(step) * 4u : kLaOob));
}

__device__ __forceinline__ int64_t row_end(const int32_t* lengths, int64_t b, int64_t seqlen) {
  if (!lengths) return seqlen;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > seqlen ? seqlen : n;
}

// The causal 16 x 16 tiles (i, j), j <= i, of a chunk's pairs of steps that a wave takes: a run of
// row i, so that the row's operand is read once, and one more tile (0, 0). Of 64 steps the waves
// take 3, 3, 3 and 1 tile (the last has the decays to do), of 32 one each but the last.
struct WaveTiles {
  int i, j0, j1;  // [j0, j1)
  bool more;
};
template <int C>
__device__ __forceinline__ WaveTiles wave_tiles(int w) {
  if constexpr (C == 64) {
    if (w == 0) return {3, 0, 3, false};
    if (w == 1) return {2, 0, 3, false};
    if (w == 2) return {1, 0, 2, true};
    return {3, 3, 4, false};
  } else {
    static_assert(C == 32, "two rows of tiles");
    if (w == 0) return {1, 0, 1, false};
    if (w == 1) return {1, 1, 2, false};
    return {0, 0, 0, w == 2};
  }
}

}  // namespace ssm
