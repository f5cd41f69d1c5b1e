// Gated RMS norm over groups of channels on gfx950 (include/ssm_norm.h): forward and gradient.
//
// Per token and group of G channels, with s = silu(z):
//   gate first   out = w v r,   v = y s,  r = 1 / sqrt(mean v^2 + eps)
//   norm first   out = w y r s,           r = 1 / sqrt(mean y^2 + eps)
// The scan writes y with time contiguous; the gate is a slice of a projection's output with
// channels contiguous, and the next projection reads channels contiguous. So a lane holds a
// square of channels by steps (16 bytes of either): a tensor of either order is read and
// written in 16-byte words and turned, where it has to be, by byte permutes within the lane.
// A workgroup holds whole groups of its steps in registers: each tensor is read once, the
// mean meets in LDS, and the result is rounded once at its store. Where every tensor has
// channels contiguous (single tokens) a lane holds one step. Groups too large for a workgroup,
// and some whose steps it would read in too small pieces, take two launches instead (Phase).
//
// Bound by memory: 3 reads and writes per element forward, 5 backward. b4, 2048 channels, 2048
// steps, bf16, y in the scan's order, z and the result in a projection's: forward 20 us (101
// MB, 5.0 TB/s, the rate of a large copy), gradient 44.4 us (168 MB, 3.8 TB/s) and 4.7 for the sums
// of dweight, 46.8 a call. The gradient's loads and its arithmetic (20 us, with two transcendentals
// per element) overlap in part only: a CU holds one workgroup of sixteen waves. Norm first, bf16:
// forward 23.3 us, of 18 registers spilled. Groups above 2048 channels take the gradient's two
// launches, which read its inputs twice (4096 channels, 1024 steps: 56.6 us a call).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_launch.h"
#include "device_block.h"

namespace ssm {
namespace {

struct Tensor {
  const void* p;
  int64_t b, c, t;  // strides in elements
  int chan;         // channels contiguous
};

struct NormParams {
  Tensor y, z, out, dout, dy, dz;
  const float* weight;
  float* rstd;
  int64_t rb, rg, rt;  // strides of rstd: batch row, group, step
  float* part;  // [batch * tiles][dim]
  float* split;  // [batch][groups][cblocks][seqlen]: sums over each block of channels
  float eps, inv_g;
  int batch, groups, g, seqlen;
  int lanes_log2;
  uint32_t tiles, cblocks, total;
};

// The words of a lane's square of CV = 16 bytes of channels by kSteps steps: one per channel, of
// its steps, when kSteps > 1; one word of channels when kSteps is 1.
template <typename Elem, int kSteps>
struct Square {
  static constexpr int CV = Vec<Elem>::kN;
  static constexpr int kWords = kSteps > 1 ? CV : 1;
  static constexpr int kSize = kSteps > 1 ? kSteps : CV;  // elements of a word
  using Word = Dwords<kSize * int(sizeof(Elem)) / 4>;
  Word w[kWords];
  __device__ __forceinline__ float at(int c, int t) const {
    return kSteps > 1 ? few_elem<Elem>(w[kSteps > 1 ? c : 0], t) : few_elem<Elem>(w[0], c);
  }
};

// Makes the compiler take the words as new, so that what was computed from them before is not
// held across a reduction (what is to be held, the gate's sigmoids, is held by name).
template <int N>
__device__ __forceinline__ void forget_word(Dwords<N>& w) {
  uint32_t v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = w.w[i];
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
#pragma unroll
  for (int i = 0; i < N; ++i) w.w[i] = v[i];
}
template <typename Elem, int kSteps>
__device__ __forceinline__ void forget(Square<Elem, kSteps>& s) {
#pragma unroll
  for (int i = 0; i < Square<Elem, kSteps>::kWords; ++i) forget_word(s.w[i]);
}

// kSteps words of CV channels turned into CV words of kSteps steps, and back.
template <typename Elem, int kSteps>
__device__ __forceinline__ void turn(const Dwords<4> (&rows)[kSteps], Square<Elem, kSteps>& s) {
  constexpr int CV = Vec<Elem>::kN;
#pragma unroll
  for (int c = 0; c < CV; ++c) {
    if constexpr (sizeof(Elem) == 4) {
#pragma unroll
      for (int t = 0; t < kSteps; ++t) s.w[c].w[t] = rows[t].w[c];
    } else {
#pragma unroll
      for (int q = 0; q < kSteps / 2; ++q)  // halves c of rows 2q and 2q + 1
        s.w[c].w[q] = __builtin_amdgcn_perm(rows[2 * q + 1].w[c / 2], rows[2 * q].w[c / 2],
                                            (c & 1) ? 0x07060302u : 0x05040100u);
    }
  }
}

template <typename Elem, int kSteps>
__device__ __forceinline__ void turn_back(const Square<Elem, kSteps>& s, Dwords<4> (&rows)[kSteps]) {
#pragma unroll
  for (int t = 0; t < kSteps; ++t) {
    if constexpr (sizeof(Elem) == 4) {
#pragma unroll
      for (int c = 0; c < 4; ++c) rows[t].w[c] = s.w[c].w[t];
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)  // halves t of channels 2q and 2q + 1
        rows[t].w[q] = __builtin_amdgcn_perm(s.w[2 * q + 1].w[t / 2], s.w[2 * q].w[t / 2],
                                             (t & 1) ? 0x07060302u : 0x05040100u);
    }
  }
}

// n (of C) elements from p on as dwords, zeros past them; and back.
template <typename Elem, int C>
__device__ __forceinline__ void load_part(const Elem* p, int n, Dwords<C * int(sizeof(Elem)) / 4>& d) {
  float v[C];
  load_few<Elem, C>(p, n, v);
  pack_few<Elem, C>(v, d);
}
template <typename Elem, int C>
__device__ __forceinline__ void store_part(Elem* p, int n, const Dwords<C * int(sizeof(Elem)) / 4>& d) {
  float v[C];
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = few_elem<Elem>(d, i);
  store_few<Elem, C>(p, n, v);
}

// d moved down by k elements (zeros come in at the top).
template <typename Elem, int N>
__device__ __forceinline__ void move_down(Dwords<N>& d, int k) {
  const int dwords = sizeof(Elem) == 2 ? k >> 1 : k;
#pragma unroll
  for (int s = 1; s < N; s *= 2) {
    const bool on = (dwords & s) != 0;
#pragma unroll
    for (int i = 0; i < N; ++i) d.w[i] = on ? (i + s < N ? d.w[i + s < N ? i + s : 0] : 0u) : d.w[i];
  }
  if constexpr (sizeof(Elem) == 2) {
    const bool on = (k & 1) != 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t above = i + 1 < N ? d.w[i + 1 < N ? i + 1 : 0] : 0u;
      d.w[i] = on ? (d.w[i] >> 16) | (above << 16) : d.w[i];
    }
  }
}

// N words `pitch` apart from p on, of which the first n (0 < n) exist, and of each its first nv (0 <
// nv) of kSize elements, zeros for the rest. What does not exist is not read: a word past n is
// the last one again, and each is read from kSize - nv elements further down, which exist, and
// moved. No branch around a load, so one trip to memory for all.
template <typename Elem, int kSize, int N>
__device__ __forceinline__ void load_edge(const Elem* p, int64_t pitch, int n, int nv,
                                          Dwords<kSize * int(sizeof(Elem)) / 4> (&d)[N]) {
  const int k = kSize - nv;
#pragma unroll
  for (int i = 0; i < N; ++i)
    d[i] = *reinterpret_cast<const Dwords<kSize * int(sizeof(Elem)) / 4>*>(p - k + (i < n ? i : n - 1) * pitch);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    move_down<Elem>(d[i], k);
#pragma unroll
    for (uint32_t& w : d[i].w) w = i < n ? w : 0u;
  }
}

// The square at (b, channel c0, step t0): nc channels and nt steps of it exist (<= 0: none), zeros
// for the rest. Whole squares take straight-line loads of whole words; those that the end of the
// group or the sequence cuts too, if either is as long as a word; the others go word by word.
template <typename Elem, int kSteps>
__device__ __forceinline__ void load_square(const NormParams& p, const Tensor& x, int b, int64_t c0, int64_t t0,
                                            int nc, int nt, Square<Elem, kSteps>& s) {
  using Sq = Square<Elem, kSteps>;
  constexpr int CV = Sq::CV;
  const Elem* at = static_cast<const Elem*>(x.p) + b * x.b + c0 * x.c + t0 * x.t;
  if constexpr (kSteps == 1) {
    load_part<Elem, CV>(at, nt > 0 ? nc : 0, s.w[0]);
  } else if (x.chan) {
    Dwords<4> rows[kSteps];
    if (nc == CV && nt == kSteps) {
#pragma unroll
      for (int t = 0; t < kSteps; ++t) rows[t] = *reinterpret_cast<const Dwords<4>*>(at + t * x.t);
    } else if (p.g >= CV && nc > 0 && nt > 0) {
      load_edge<Elem, CV, kSteps>(at, x.t, nt, nc, rows);
    } else {
#pragma unroll
      for (int t = 0; t < kSteps; ++t) load_part<Elem, CV>(at + t * x.t, t < nt ? nc : 0, rows[t]);
    }
    turn<Elem, kSteps>(rows, s);
  } else if (nc == CV && nt == kSteps) {
#pragma unroll
    for (int c = 0; c < CV; ++c) s.w[c] = *reinterpret_cast<const typename Sq::Word*>(at + c * x.c);
  } else if (p.seqlen >= kSteps && nc > 0 && nt > 0) {
    load_edge<Elem, kSteps, CV>(at, x.c, nc, nt, s.w);
  } else {
#pragma unroll
    for (int c = 0; c < CV; ++c) load_part<Elem, kSteps>(at + c * x.c, c < nc ? nt : 0, s.w[c]);
  }
}

template <typename Elem, int kSteps>
__device__ __forceinline__ void store_square(const Tensor& x, int b, int64_t c0, int64_t t0, int nc, int nt,
                                             const Square<Elem, kSteps>& s) {
  using Sq = Square<Elem, kSteps>;
  constexpr int CV = Sq::CV;
  Elem* p = static_cast<Elem*>(const_cast<void*>(x.p)) + b * x.b + c0 * x.c + t0 * x.t;
  if constexpr (kSteps == 1) {
    store_part<Elem, CV>(p, nt > 0 ? nc : 0, s.w[0]);
  } else if (x.chan) {
    Dwords<4> rows[kSteps];
    turn_back<Elem, kSteps>(s, rows);
    if (nc == CV && nt == kSteps) {
#pragma unroll
      for (int t = 0; t < kSteps; ++t) store_stream(p + t * x.t, rows[t]);
    } else {
#pragma unroll
      for (int t = 0; t < kSteps; ++t) store_part<Elem, CV>(p + t * x.t, t < nt ? nc : 0, rows[t]);
    }
  } else if (nc == CV && nt == kSteps) {
#pragma unroll
    for (int c = 0; c < CV; ++c) *reinterpret_cast<typename Sq::Word*>(p + c * x.c) = s.w[c];
  } else {
#pragma unroll
    for (int c = 0; c < CV; ++c) store_part<Elem, kSteps>(p + c * x.c, c < nc ? nt : 0, s.w[c]);
  }
}

// Channel c's steps v rounded into the square, channel by channel so that few values are live
// in fp32 (one word of all channels, with one step, is formed when the last has come: `row`
// gathers it).
template <typename Elem, int kSteps>
__device__ __forceinline__ void put(Square<Elem, kSteps>& s, int c, const float (&v)[kSteps],
                                    float (&row)[Vec<Elem>::kN]) {
  constexpr int CV = Vec<Elem>::kN;
  if constexpr (kSteps > 1) {
    pack_few<Elem, kSteps>(v, s.w[c]);
  } else {
    row[c] = v[0];
    if (c == CV - 1) pack_few<Elem, CV>(row, s.w[0]);
  }
}

// Without a gate, gate first, norm first.
enum Mode { kNoGate = 0, kGateFirst = 1, kNormFirst = 2 };

// Where a lane is in its wave: its low bits along time, the 2^lg lanes of the others along the
// channels. Lanes next to each other then read on in a tensor with steps contiguous, and its
// accesses, of which each channel needs its own, are a quarter in number (the gradient at b4,
// 2048 channels, 2048 steps: 46 -> 44 us with y so ordered, 53 -> 41 with all so ordered;
// tensors with channels contiguous lose nothing that shows).
struct LaneMap {
  int lg;
  __device__ __forceinline__ int time() const { return threadIdx.x & ((64 >> lg) - 1); }
  __device__ __forceinline__ int channel() const { return (threadIdx.x & 63) >> (6 - lg); }
  __device__ __forceinline__ bool along_time(int bit) const { return bit < 6 - lg; }
};

template <int kBit, int N>
__device__ __forceinline__ void add_across(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (kBit == 0)
      v[i] = dpp_add<0xB1>(v[i]);  // quad_perm 1,0,3,2
    else if constexpr (kBit == 1)
      v[i] = dpp_add<0x4E>(v[i]);  // quad_perm 2,3,0,1
    else if constexpr (kBit == 3)
      v[i] = dpp_add<0x128>(v[i]);  // row_ror:8
    else
      v[i] += __shfl_xor(v[i], 1 << kBit, 64);
  }
}

// Each v[i] summed over the lanes along the channels (or, kTime, along time), in every lane.
template <bool kTime, int N>
__device__ __forceinline__ void sum_wave(float (&v)[N], const LaneMap& m) {
  if (m.along_time(0) == kTime) add_across<0>(v);
  if (m.along_time(1) == kTime) add_across<1>(v);
  if (m.along_time(2) == kTime) add_across<2>(v);
  if (m.along_time(3) == kTime) add_across<3>(v);
  if (m.along_time(4) == kTime) add_across<4>(v);
  if (m.along_time(5) == kTime) add_across<5>(v);
}

// ... and over the workgroup's waves, in wave order: buf holds waves x lanes-along-time x N.
template <int N>
__device__ __forceinline__ void sum_group(float (&v)[N], const LaneMap& m, float* buf) {
  sum_wave<false>(v, m);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return;
  const int wave = threadIdx.x >> 6, tb = m.time(), times = 64 >> m.lg;
  if (m.channel() == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[(wave * times + tb) * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int w = 0; w < waves; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += buf[(w * times + tb) * N + i];
}

// Where a workgroup's lanes are; consecutive tiles, which share cache lines of the time-ordered
// tensors, go to one XCD.
struct Place {
  int b, grp, cb, tile, nt;
  int64_t t0, c0;  // first step; first channel within the group
  LaneMap map;
};

template <typename Elem, int kSteps>
__device__ __forceinline__ Place place_of(const NormParams& p) {
  constexpr int CV = Vec<Elem>::kN;
  const uint32_t id = xcd_order(blockIdx.x, p.total);
  const int waves = blockDim.x >> 6, wave = threadIdx.x >> 6;
  Place a;
  a.map = LaneMap{p.lanes_log2};
  a.tile = int(id % p.tiles);
  uint32_t rest = id / p.tiles;
  a.cb = int(rest % p.cblocks);
  rest /= p.cblocks;
  a.grp = int(rest % uint32_t(p.groups));
  a.b = int(rest / uint32_t(p.groups));
  a.t0 = (int64_t(a.tile) * (64 >> p.lanes_log2) + a.map.time()) * kSteps;
  a.nt = a.t0 >= p.seqlen ? 0 : p.seqlen - a.t0 < kSteps ? int(p.seqlen - a.t0) : kSteps;
  a.c0 = ((int64_t(a.cb * waves + wave) << p.lanes_log2) + a.map.channel()) * CV;
  return a;
}

// What a launch does of a norm whose sums run over a group: all of it, a workgroup holding whole
// groups; or, in two launches, a workgroup holding a block of a group's channels, first the sums
// over its block, then the rest from all blocks' sums.
enum Phase { kWhole = 0, kSums = 1, kApply = 2 };

// A workgroup's sums over its block of channels to memory, one per step.
template <int N>
__device__ __forceinline__ void store_sums(const NormParams& p, const Place& a, const float (&v)[N]) {
  if ((threadIdx.x >> 6) != 0 || a.map.channel() != 0) return;
  float* row = p.split + ((int64_t(a.b) * p.groups + a.grp) * p.cblocks + a.cb) * p.seqlen + a.t0;
#pragma unroll
  for (int t = 0; t < N; ++t)
    if (t < a.nt) row[t] = v[t];
}

// The sums of all blocks of a group, for this lane's steps, in block order within each slice of
// the workgroup and then over the slices. buf: blockDim floats.
template <int N>
__device__ __forceinline__ void load_sums(const NormParams& p, const Place& a, float (&v)[N], float* buf) {
  const int span = (64 >> p.lanes_log2) * N;  // the workgroup's steps: at most 64, a power of two
  const int at = threadIdx.x & (span - 1), slice = threadIdx.x / span, slices = blockDim.x / span;
  const int64_t t = int64_t(a.tile) * span + at;
  const float* col = p.split + (int64_t(a.b) * p.groups + a.grp) * p.cblocks * p.seqlen + t;
  float sum = 0.0f;
  if (t < p.seqlen)
    for (uint32_t k = slice; k < p.cblocks; k += slices) sum += col[int64_t(k) * p.seqlen];
  buf[threadIdx.x] = sum;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int k = 0; k < slices; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += buf[k * span + a.map.time() * N + i];
}

template <int CV>
__device__ __forceinline__ int channels_left(const NormParams& p, int64_t c0) {
  return c0 >= p.g ? 0 : p.g - c0 < CV ? int(p.g - c0) : CV;
}

// ---------------------------------------------------------------- forward
//
template <typename Elem, int kSteps, int kPhase, int kMode>
__global__ __launch_bounds__(64 * kNormMostWaves) void norm_fwd_kernel(NormParams p) {
  constexpr int CV = Vec<Elem>::kN;
  extern __shared__ float buf[];
  const Place a = place_of<Elem, kSteps>(p);
  const int64_t base = int64_t(a.grp) * p.g + a.c0;
  const int nc = channels_left<CV>(p, a.c0);
  Square<Elem, kSteps> y, z;
  float q[CV][kSteps], sum[kSteps];  // q: y s, the result but for w r
#pragma unroll
  for (int t = 0; t < kSteps; ++t) sum[t] = 0.0f;
  load_square<Elem, kSteps>(p, p.y, a.b, base, a.t0, nc, a.nt, y);
  if constexpr (kMode == kGateFirst || (kMode == kNormFirst && kPhase != kSums))
    load_square<Elem, kSteps>(p, p.z, a.b, base, a.t0, nc, a.nt, z);
#pragma unroll
  for (int c = 0; c < CV; ++c) {
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const float v = y.at(c, t);
      if constexpr (kMode == kGateFirst || (kMode == kNormFirst && kPhase != kSums))
        q[c][t] = v * silu_f(z.at(c, t));
      else
        q[c][t] = v;
      const float n = kMode == kNormFirst ? v : q[c][t];
      if constexpr (kPhase != kApply) sum[t] = __builtin_fmaf(n, n, sum[t]);
    }
    // A channel's words go out of use as its values come into it, if the channels are not
    // interleaved.
    if constexpr (kSteps > 1) __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (kPhase == kApply)
    load_sums<kSteps>(p, a, sum, buf);
  else
    sum_group<kSteps>(sum, a.map, buf);
  if constexpr (kPhase == kSums) {
    store_sums<kSteps>(p, a, sum);
    return;
  }
  float r[kSteps], w[CV], row[CV];
#pragma unroll
  for (int t = 0; t < kSteps; ++t) r[t] = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[t], p.inv_g, p.eps));
  if (p.rstd && a.c0 == 0) {
#pragma unroll
    for (int t = 0; t < kSteps; ++t)
      if (t < a.nt) p.rstd[a.b * p.rb + a.grp * p.rg + (a.t0 + t) * p.rt] = r[t];
  }
  load_run<float, CV>(p.weight + base, nc, w);
  Square<Elem, kSteps> o;
#pragma unroll
  for (int c = 0; c < CV; ++c) {
    float v[kSteps];
#pragma unroll
    for (int t = 0; t < kSteps; ++t) v[t] = q[c][t] * (r[t] * w[c]);
    put<Elem, kSteps>(o, c, v, row);
  }
  store_square<Elem, kSteps>(p.out, a.b, base, a.t0, nc, a.nt, o);
}

// ---------------------------------------------------------------- backward
//
// gate first: A = w dout;    n = v r, k = r S / G, S = sum_G A v; dv = r (A - n k); dy = dv s; dz = dv y s'
// norm first: A = w dout s;  n = y r, k = r S / G, S = sum_G A y; dy = r (A - n k); dz = w dout n s'
// n is of order one and k of A's, so no power of r but the first is formed: r^3 alone would leave
// float32's range for values of 1e13 (and 1e-13, eps 0), long before their squares do.
// dweight = sum over tokens of dout (s) times the normed value; per workgroup and channel
// here, over workgroups by a second launch in a fixed order.
template <typename Elem, int kSteps, int kPhase, int kMode>
__global__ __launch_bounds__(64 * kNormMostWaves) void norm_bwd_kernel(NormParams p) {
  constexpr int CV = Vec<Elem>::kN;
  extern __shared__ float buf[];
  const Place a = place_of<Elem, kSteps>(p);
  const int64_t base = int64_t(a.grp) * p.g + a.c0;
  const int nc = channels_left<CV>(p, a.c0);
  Square<Elem, kSteps> y, z, g;
  float w[CV], sum[kSteps], r[kSteps], sigma[CV][kSteps];
  load_square<Elem, kSteps>(p, p.y, a.b, base, a.t0, nc, a.nt, y);
  if constexpr (kMode != kNoGate) load_square<Elem, kSteps>(p, p.z, a.b, base, a.t0, nc, a.nt, z);
  load_square<Elem, kSteps>(p, p.dout, a.b, base, a.t0, nc, a.nt, g);
  load_run<float, CV>(p.weight + base, nc, w);
#pragma unroll
  for (int t = 0; t < kSteps; ++t) {
    sum[t] = 0.0f;
    r[t] = t < a.nt ? p.rstd[a.b * p.rb + a.grp * p.rg + (a.t0 + t) * p.rt] : 0.0f;
  }
  if constexpr (kPhase == kApply) {
    load_sums<kSteps>(p, a, sum, buf);
  } else {
    // sum_G A v: w dout y s either way
#pragma unroll
    for (int c = 0; c < CV; ++c) {
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        float v = y.at(c, t);
        if constexpr (kMode != kNoGate) {
          const float zv = z.at(c, t), sg = sigmoid_f(zv);
          sigma[c][t] = sg;
          v *= zv * sg;
        }
        sum[t] = __builtin_fmaf(w[c] * g.at(c, t), v, sum[t]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    sum_group<kSteps>(sum, a.map, buf);
  }
  if constexpr (kPhase == kSums) {
    store_sums<kSteps>(p, a, sum);
    return;
  }
  float k[kSteps];
#pragma unroll
  for (int t = 0; t < kSteps; ++t) k[t] = r[t] * (sum[t] * p.inv_g);
  forget<Elem, kSteps>(y);
  forget<Elem, kSteps>(g);
  if constexpr (kMode != kNoGate) forget<Elem, kSteps>(z);

  float dw[CV], row_y[CV], row_z[CV];
  Square<Elem, kSteps> dys, dzs;
#pragma unroll
  for (int c = 0; c < CV; ++c) {
    float dy[kSteps], dz[kSteps];
    dw[c] = 0.0f;
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const float yv = y.at(c, t), gv = g.at(c, t);
      float s = 1.0f, ds = 0.0f;
      if constexpr (kMode != kNoGate) {
        const float zv = z.at(c, t), sg = kPhase == kWhole ? sigma[c][t] : sigmoid_f(zv);
        s = zv * sg;
        ds = __builtin_fmaf(s, 1.0f - sg, sg);
      }
      const float wg = w[c] * gv;
      if constexpr (kMode == kNormFirst) {
        const float n = yv * r[t];
        dw[c] = __builtin_fmaf(gv, n * s, dw[c]);
        dy[t] = r[t] * __builtin_fmaf(-n, k[t], wg * s);
        dz[t] = wg * (n * ds);
      } else {
        const float n = (kMode == kNoGate ? yv : yv * s) * r[t];
        dw[c] = __builtin_fmaf(gv, n, dw[c]);
        const float dv = r[t] * __builtin_fmaf(-n, k[t], wg);
        dy[t] = dv * s;
        dz[t] = dv * (yv * ds);
      }
    }
    put<Elem, kSteps>(dys, c, dy, row_y);
    if constexpr (kMode != kNoGate) put<Elem, kSteps>(dzs, c, dz, row_z);
    // A channel's words go out of use as its gradients' words come into it, if the channels
    // are not interleaved (nor its sums put off).
    asm volatile("" : "+v"(dw[c]));
    forget_word(dys.w[c]);
    if constexpr (kMode != kNoGate) forget_word(dzs.w[c]);
    __builtin_amdgcn_sched_barrier(0);
  }
  store_square<Elem, kSteps>(p.dy, a.b, base, a.t0, nc, a.nt, dys);
  if constexpr (kMode != kNoGate) store_square<Elem, kSteps>(p.dz, a.b, base, a.t0, nc, a.nt, dzs);
  // over the lanes along time, then one store per channel
  sum_wave<true>(dw, a.map);
  if (a.map.time() == 0)
    store_run<float, CV>(p.part + (int64_t(a.b) * p.tiles + a.tile) * (int64_t(p.groups) * p.g) + base, nc, dw);
}

__global__ __launch_bounds__(kReduceCols* kNormReduceSlices) void norm_bwd_reduce(const float* part, float* dweight,
                                                                              int64_t rows, int64_t cols) {
  __shared__ float buf[kNormReduceSlices][kReduceCols + 1];
  const int64_t col = int64_t(blockIdx.x) * kReduceCols + threadIdx.x % kReduceCols;
  const float a = sum_rows<kReduceCols, kNormReduceSlices>(part, rows, cols, col, buf);
  if (threadIdx.x < kReduceCols && col < cols) dweight[col] = a;
}

Tensor tensor_of(const View& v) {
  return Tensor{v.p, v.s.batch, v.s.channel, v.s.step, v.order == Order::Channel ? 1 : 0};
}

NormParams params_of(const NormArgs& a, const NormShape& s) {
  NormParams p{};
  p.y = tensor_of(a.y);
  p.z = tensor_of(a.z);
  p.out = tensor_of(a.out);
  p.dout = tensor_of(a.dout);
  p.dy = tensor_of(a.dy);
  p.dz = tensor_of(a.dz);
  p.weight = a.weight;
  p.rstd = a.rstd;
  p.rb = a.rs.batch;
  p.rg = a.rs.channel;
  p.rt = a.rs.step;
  p.part = a.workspace;
  p.eps = a.eps;
  p.g = int(a.dim / a.groups);
  p.inv_g = 1.0f / float(p.g);
  p.batch = int(a.batch);
  p.groups = int(a.groups);
  p.seqlen = int(a.seqlen);
  p.lanes_log2 = s.lanes_log2;
  p.tiles = uint32_t(s.tiles);
  p.cblocks = uint32_t(s.cblocks);
  p.total = uint32_t(s.tiles * s.cblocks * a.groups * a.batch);
  return p;
}

template <typename Elem, int kSteps, int kPhase, int kMode>
void launch(const NormParams& p, const NormShape& s, bool backward, hipStream_t st) {
  constexpr int io = sizeof(Elem) == 2 ? int(Io::BF16) : int(Io::F32);
  const dim3 grid(p.total), block(64 * s.waves);
  const size_t lds = kPhase == kApply ? size_t(64) * s.waves * 4
                                      : size_t(s.waves) * (64 >> s.lanes_log2) * kSteps * 4;
  if constexpr (kSteps == kNormBwdSteps[io]) {
    if (backward) hipLaunchKernelGGL((norm_bwd_kernel<Elem, kSteps, kPhase, kMode>), grid, block, lds, st, p);
  }
  if constexpr (kSteps == 1 || kSteps == kNormFwdSteps[io]) {
    if (!backward) hipLaunchKernelGGL((norm_fwd_kernel<Elem, kSteps, kPhase, kMode>), grid, block, lds, st, p);
  }
}

template <typename Elem, int kSteps, int kPhase>
void run_phase(const NormParams& p, const NormShape& s, bool backward, bool norm_first, hipStream_t st) {
  if (!p.z.p)
    launch<Elem, kSteps, kPhase, kNoGate>(p, s, backward, st);
  else if (norm_first)
    launch<Elem, kSteps, kPhase, kNormFirst>(p, s, backward, st);
  else
    launch<Elem, kSteps, kPhase, kGateFirst>(p, s, backward, st);
}

template <typename Elem, int kSteps>
void run_steps(const NormParams& p, const NormShape& s, bool backward, bool norm_first, hipStream_t st) {
  if (!s.split) return run_phase<Elem, kSteps, kWhole>(p, s, backward, norm_first, st);
  if constexpr (kSteps > 1) {
    run_phase<Elem, kSteps, kSums>(p, s, backward, norm_first, st);
    run_phase<Elem, kSteps, kApply>(p, s, backward, norm_first, st);
  }
}

template <typename Elem>
void run(const NormParams& p, const NormShape& s, bool backward, bool norm_first, hipStream_t st) {
  constexpr int io = sizeof(Elem) == 2 ? int(Io::BF16) : int(Io::F32);
  if (backward)
    run_steps<Elem, kNormBwdSteps[io]>(p, s, true, norm_first, st);
  else if (s.steps == 1)
    run_steps<Elem, 1>(p, s, false, norm_first, st);
  else
    run_steps<Elem, kNormFwdSteps[io]>(p, s, false, norm_first, st);
}

}  // namespace

int launch_norm_fwd(const NormArgs& a, void* stream) {
  const NormShape s = norm_fwd_shape(a);
  NormParams p = params_of(a, s);
  p.split = a.workspace;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.io == Io::BF16)
    run<uint16_t>(p, s, false, a.norm_first, st);
  else
    run<float>(p, s, false, a.norm_first, st);
  return int(hipGetLastError());
}

int launch_norm_bwd(const NormArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  int64_t rows = 0;
  if (a.batch > 0 && a.seqlen > 0) {
    const NormShape s = norm_bwd_shape(a);
    NormParams p = params_of(a, s);
    rows = norm_partials(a.batch, s);
    p.split = a.workspace + rows * a.dim;
    if (a.io == Io::BF16)
      run<uint16_t>(p, s, true, a.norm_first, st);
    else
      run<float>(p, s, true, a.norm_first, st);
    const int err = int(hipGetLastError());
    if (err) return err;
  }
  hipLaunchKernelGGL(norm_bwd_reduce, dim3(unsigned(reduce_groups(a.dim))),
                     dim3(kReduceCols * kNormReduceSlices), 0, st, a.workspace, a.dweight, rows, a.dim);
  return int(hipGetLastError());
}

}  // namespace ssm
