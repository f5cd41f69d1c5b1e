// Short causal convolution over time on gfx950 (include/ssm_conv.h): forward, gradient and
// single-token step.
//
// Per batch row b and channel d, with e the row's inputs behind its initial state (place m of
// e is step m - (W - 1)): p_t = bias + sum_k w[k] e[t + k], out_t = p_t or silu(p_t).
//
// A lane owns kConvSteps = 8 consecutive steps of a channel, so that a step's window is in
// registers and only the W - 1 inputs at a block's edge are fetched twice (or taken from the
// neighbouring lane). Two orders of x in memory:
//   time     runs of steps: a lane holds one channel's 8 steps, lanes lie along time;
//   channel  runs of channels (a slice of a projection's output): a lane holds 4 channels by 8
//            steps, loads one word of channels per step and stores one run of steps per
//            channel, which turns the order through registers alone. A wave covers 64
//            channels by 32 steps, a workgroup 128 steps.
// Sums are fp32; a result is rounded once, at its store. A row's steps at and behind its
// length are not read, and its outputs there are zeros.
//
// b4, 2304 channels, 2048 steps, bf16 (75 MB in and out, 12 us by a library copy of that size):
// 14.7 us channel order by the kernel trace; 14.9 and 15.6 (time order) a call. What that took: no branch
// around a load (23 -> 16 us, with the weights of a workgroup in LDS instead of a load per
// channel that is waited for), index arithmetic of 32 bits (time order 20 -> 16: it was VALU
// bound), stores past L2 (1 us). Eight channels a lane 17.7 us, sixteen-channel waves 28 us.
// The gradient (113 MB): 30.6 us channel order by the trace, of which the VALU needs 21 (a sigmoid
// for 11 steps of each 8), and 4.8 the second launch; 33.4 and 31.6 (time order) a call. 43 us with
// workgroups in plain order, where an XCD's tiles all lie at one offset of the 4096-byte rows and
// so in two of its L2's channels. fp32, channel order: 50.5 a call (227 MB).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_launch.h"
#include "device_block.h"

namespace ssm {
namespace {

constexpr int S = kConvSteps;
constexpr int kThreads = 64 * kConvWaves;
constexpr int CW = kConvWaveChannels;

struct ConvParams {
  const void* x;
  int64_t xb, xc, xt;
  const float* weight;
  const float* bias;
  const void* initial;
  const int32_t* lengths;
  void* out;
  void* final_state;
  const void* dout;
  const void* dfinal;
  void* dx;
  int64_t dxb, dxc, dxt;
  void* dinitial;
  float* part;       // [batch * runs][dim][W + 1]
  uint32_t dim, seqlen;
  int silu;
  uint32_t waves;    // time order: waves with work, per batch row
  uint32_t tiles;    // runs of steps per row
  int lanes_log2;    // time order: lanes along a row
};

// The grid's second axis is the batch row.
__device__ __forceinline__ uint32_t row_length(const ConvParams& p, int b) {
  if (!p.lengths) return p.seqlen;
  const int n = p.lengths[b];
  return n < 0 ? 0 : uint32_t(n) > p.seqlen ? p.seqlen : uint32_t(n);
}

// Steps of a row from t0 on, before `end`.
__device__ __forceinline__ int steps_left(uint32_t end, uint32_t t0) { return t0 < end ? int(end - t0) : 0; }

template <int W>
__device__ __forceinline__ void load_weights(const ConvParams& p, uint32_t d, float (&w)[W], float& bias) {
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = p.weight[int64_t(d) * W + k];
  bias = p.bias ? p.bias[d] : 0.0f;
}

// Place m of e, in fp32: the initial state for m < W - 1 (zero without one), x at step m - (W - 1).
template <typename Elem, int W>
__device__ __forceinline__ Elem place(const ConvParams& p, const Elem* xrow, int64_t row, int64_t m) {
  if (m >= W - 1) return xrow[(m - (W - 1)) * p.xt];
  if (!p.initial) return Elem(0);
  return static_cast<const Elem*>(p.initial)[row * (W - 1) + m];
}

// The last W - 1 inputs before the row's end (one lane per row).
template <typename Elem, int W>
__device__ __forceinline__ void store_final(const ConvParams& p, const Elem* xrow, int64_t row, uint32_t len) {
  Elem* f = static_cast<Elem*>(p.final_state) + row * (W - 1);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) f[k] = place<Elem, W>(p, xrow, row, int64_t(len) + k);
}

// e[0 .. W - 2] of a row's first steps.
template <typename Elem, int W, int E>
__device__ __forceinline__ void load_initial(const ConvParams& p, int64_t row, float (&e)[E]) {
#pragma unroll
  for (int i = 0; i < W - 1; ++i)
    e[i] = p.initial ? widen<Elem>(static_cast<const Elem*>(p.initial)[row * (W - 1) + i]) : 0.0f;
}

// e[0 .. W - 2] of a block that starts at step t0 > 0 of a row of contiguous steps (t0 >= 4).
template <typename Elem, int W, int E>
__device__ __forceinline__ void load_left(const Elem* xrow, uint32_t t0, uint32_t len, float (&e)[E]) {
  float v[4];
  load_few<Elem, 4>(xrow + t0 - 4, steps_left(len, t0 - 4), v);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) e[i] = v[4 - (W - 1) + i];
}

template <int W, int E>
__device__ __forceinline__ float window(const float (&w)[W], float bias, const float (&e)[E], int i) {
  float acc = bias;
#pragma unroll
  for (int k = 0; k < W; ++k) acc = __builtin_fmaf(w[k], e[i + k], acc);
  return acc;
}

// The S outputs of a block, zeros from the n-th on.
template <int W>
__device__ __forceinline__ void conv_block(const float (&w)[W], float bias, bool silu,
                                           const float (&e)[S + W - 1], int n, float (&o)[S]) {
#pragma unroll
  for (int i = 0; i < S; ++i) o[i] = window<W>(w, bias, e, i);
  if (silu) {
#pragma unroll
    for (int i = 0; i < S; ++i) o[i] = silu_f(o[i]);
  }
  if (n < S) {
#pragma unroll
    for (int i = 0; i < S; ++i) o[i] = i < n ? o[i] : 0.0f;
  }
}

// Where a lane of the time-ordered kernels is: 2^lanes_log2 lanes along a row.
struct TimeLane {
  uint32_t d, run, j;
  bool live;
};

__device__ __forceinline__ TimeLane time_lane(const ConvParams& p) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * kConvWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t group = wave / p.tiles;
  TimeLane a;
  a.run = wave - group * p.tiles;
  a.j = lane & ((1u << p.lanes_log2) - 1);
  a.d = (group << (6 - p.lanes_log2)) + (lane >> p.lanes_log2);
  a.live = wave < p.waves && a.d < p.dim;
  return a;
}

// ---------------------------------------------------------------- forward, time order

// A wave takes T consecutive tiles of its rows, their loads in flight together.
template <typename Elem, int W, int T>
__global__ __launch_bounds__(kThreads) void conv_fwd_time(ConvParams p) {
  const TimeLane a = time_lane(p);
  if (!a.live) return;
  const int b = blockIdx.y;
  const int64_t row = int64_t(b) * p.dim + a.d;
  const uint32_t len = row_length(p, b);
  const Elem* xrow = static_cast<const Elem*>(p.x) + b * p.xb + a.d * p.xc;
  Elem* orow = static_cast<Elem*>(p.out) + row * p.seqlen;
  const uint32_t step = uint32_t(S) << p.lanes_log2, start = a.run * T * step + a.j * S;
  float w[W], bias, e[T][S + W - 1];
#pragma unroll
  for (int q = 0; q < T; ++q) {
    const uint32_t t0 = start + q * step;
    float own[S];
    load_run<Elem, S>(xrow + t0, steps_left(len, t0), own);
#pragma unroll
    for (int i = 0; i < S; ++i) e[q][W - 1 + i] = own[i];
  }
  load_weights<W>(p, a.d, w, bias);
#pragma unroll
  for (int q = 0; q < T; ++q) {
    const uint32_t t0 = start + q * step;
    // The left edge is the last steps of the lane before (of the same row, so active too).
#pragma unroll
    for (int i = 0; i < W - 1; ++i) e[q][i] = shift_up_one(e[q][S + i], 0.0f);
    if (a.j == 0) {
      if (t0 == 0)
        load_initial<Elem, W>(p, row, e[q]);
      else
        load_left<Elem, W>(xrow, t0, len, e[q]);
    }
    float o[S];
    conv_block<W>(w, bias, p.silu, e[q], steps_left(len, t0), o);
    store_run_stream<Elem, S>(orow + t0, steps_left(p.seqlen, t0), o);
  }
  if (p.final_state && a.run == 0 && a.j == 0) store_final<Elem, W>(p, xrow, row, len);
}

// ---------------------------------------------------------------- channel order

// Words of the steps t .. t + N - 1, of nc (> 0) channels from p's on. A step outside the row (end > 0
// is its length) takes the nearest one's word, so that the loads need no branch and what lies
// behind the row is not read: the callers replace what lies before the first step by the initial
// state and let nothing at or behind the end count. (A row of no steps takes no words; theirs are
// then what the registers held, and count as little. Stopping a workgroup behind its row's end
// ahead of its loads made whole rows 4% slower; as it is, b16, 2304 channels, 2048 steps, rows of
// a quarter to three quarters, bf16, take 40.5 us, 66.9 with their padding read.)
template <typename Elem, int CV>
using Word = Dwords<CV * int(sizeof(Elem)) / 4>;

template <typename Elem, int CV, int N>
__device__ __forceinline__ void load_rows(const Elem* p, int64_t pitch, int64_t t, uint32_t end, int nc,
                                          Word<Elem, CV> (&raw)[N]) {
  const Elem* at[N];
  if (t >= 0 && t + N <= end) {
    at[0] = p + t * pitch;
#pragma unroll
    for (int i = 1; i < N; ++i) at[i] = at[i - 1] + pitch;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      at[i] = p + (t + i < 0 ? 0 : t + i >= end ? int64_t(end) - 1 : t + i) * pitch;
  }
  if (nc >= CV) {
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = *reinterpret_cast<const Word<Elem, CV>*>(at[i]);
  } else {
    Elem e[N][CV];  // (past nc the last channel again: no branch around a load here either)
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < CV; ++c) e[i][c] = at[i][c < nc ? c : nc - 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v[CV];
#pragma unroll
      for (int c = 0; c < CV; ++c) v[c] = c < nc ? widen<Elem>(e[i][c]) : 0.0f;
      pack_few<Elem, CV>(v, raw[i]);
    }
  }
}

// Where a lane of the channel-ordered kernels is: CG lanes along channels, TB along time; a
// workgroup's waves along time.
template <int kCV>
struct ChanLane {
  static constexpr int CV = kCV;  // channels per lane
  static constexpr int CG = CW / CV;
  static constexpr int TB = 64 / CG;
  uint32_t tile, cb, cl, c0, t0;
  int b, wv, tb, nc;
};

template <int CV, bool kXcdOrder>
__device__ __forceinline__ ChanLane<CV> chan_lane(const ConvParams& p) {
  using L = ChanLane<CV>;
  const int lane = threadIdx.x & 63;
  L a;
  a.wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  a.tb = lane / L::CG;
  uint32_t in_row = blockIdx.x;
  a.b = blockIdx.y;
  if constexpr (kXcdOrder) {
    const uint32_t id = xcd_order(blockIdx.y * gridDim.x + blockIdx.x, gridDim.x * gridDim.y);
    a.b = int(id / gridDim.x);
    in_row = id - a.b * gridDim.x;
  }
  a.cb = in_row / p.tiles;
  a.tile = in_row - a.cb * p.tiles;
  a.cl = (lane % L::CG) * L::CV;
  a.c0 = a.cb * CW + a.cl;
  a.t0 = ((a.tile * kConvWaves + a.wv) * L::TB + a.tb) * S;
  a.nc = a.c0 < p.dim ? int(p.dim - a.c0) : 0;  // channels from c0 on
  return a;
}

// The weights and biases of the workgroup's channels, through LDS: every lane needs its
// channels' in turn, and a load from memory for each would be waited for each time. They are
// loaded ahead of the block's inputs (loads complete in order), so the barrier does not wait
// for those.
template <int W>
struct Weights {
  static constexpr int kPer = (CW * (W + 1) + kThreads - 1) / kThreads;
  float v[kPer];
  __device__ __forceinline__ void load(const ConvParams& p, uint32_t cb) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int i = threadIdx.x + q * kThreads;  // the weights, then the biases
      const int64_t at = i < CW * W ? int64_t(cb) * CW * W + i : int64_t(cb) * CW + (i - CW * W);
      v[q] = 0.0f;
      if (i < CW * W) {
        if (at < int64_t(p.dim) * W) v[q] = p.weight[at];
      } else if (i < CW * (W + 1) && p.bias && at < p.dim) {
        v[q] = p.bias[at];
      }
    }
  }
  __device__ __forceinline__ void stage(float (&s)[CW * (W + 1)]) const {
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (threadIdx.x + q * kThreads < CW * (W + 1)) s[threadIdx.x + q * kThreads] = v[q];
    __syncthreads();
  }
  // Channel c of the workgroup's.
  static __device__ __forceinline__ void of(const float (&s)[CW * (W + 1)], int c, float (&w)[W], float& bias) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = s[c * W + k];
    bias = s[CW * W + c];
  }
};

template <typename Elem, int W>
__global__ __launch_bounds__(kThreads) void conv_fwd_chan(ConvParams p) {
  constexpr int CV = kConvLaneChannels;
  __shared__ float sw[CW * (W + 1)];
  const ChanLane<CV> a = chan_lane<CV, false>(p);
  Weights<W> weights;
  weights.load(p, a.cb);
  const int b = a.b;
  const bool live = a.nc > 0 && a.t0 < p.seqlen;
  const Elem* xb = static_cast<const Elem*>(p.x) + b * p.xb + a.c0;
  const uint32_t len = row_length(p, b);
  Word<Elem, CV> raw[S + W - 1];
  if (live && len > 0) load_rows<Elem, CV, S + W - 1>(xb, p.xt, int64_t(a.t0) - (W - 1), len, a.nc, raw);
  weights.stage(sw);
  if (!live) return;
  const int n = steps_left(len, a.t0), all = steps_left(p.seqlen, a.t0);
  const int64_t row0 = int64_t(b) * p.dim + a.c0;
  Elem* orow = static_cast<Elem*>(p.out) + row0 * p.seqlen + a.t0;
  const bool first = a.tile == 0 && a.wv == 0;  // of the wave; its lanes of tb 0 start the row
#pragma unroll
  for (int c = 0; c < CV; ++c) {
    float w[W], bias, e[S + W - 1], o[S];
    Weights<W>::of(sw, a.cl + c, w, bias);
#pragma unroll
    for (int i = 0; i < S + W - 1; ++i) e[i] = few_elem<Elem>(raw[i], c);
    if (first && a.tb == 0 && c < a.nc) load_initial<Elem, W>(p, row0 + c, e);
    conv_block<W>(w, bias, p.silu, e, n, o);
    if (c < a.nc) store_run_stream<Elem, S>(orow, all, o);
    orow += p.seqlen;
  }
  if (p.final_state && first && a.tb == 0) {
    for (int c = 0; c < CV; ++c)
      if (c < a.nc) store_final<Elem, W>(p, xb + c, row0 + c, len);
  }
}

// ---------------------------------------------------------------- backward
//
// dp_t = dout_t silu'(p_t) (dout_t without silu, 0 at and behind the row's length);
// dx_t = sum_k w[k] dp_{t + W - 1 - k}, plus dfinal of the last W - 1 steps;
// dw[k] = sum_{b,t} dp_t e[t + k], dbias = sum_{b,t} dp_t.
// A lane forms dp of its 8 steps and of the W - 1 behind them. dw and dbias are summed per
// lane, over the workgroup's lanes, and over workgroups by a second launch in a fixed order.

// From e[0 .. S + 2 (W - 1)) and dout g[0 .. S + W - 1) of the steps t0 on: dx of the S steps
// and this lane's sums.
template <int W>
__device__ __forceinline__ void conv_grad_block(const float (&w)[W], float bias, bool silu,
                                                const float (&e)[S + 2 * (W - 1)],
                                                const float (&g)[S + W - 1], float (&dx)[S],
                                                float (&dw)[W + 1]) {
  float dp[S + W - 1];
#pragma unroll
  for (int i = 0; i < S + W - 1; ++i) dp[i] = g[i];
  if (silu) {
#pragma unroll
    for (int i = 0; i < S + W - 1; ++i) dp[i] *= silu_grad_f(window<W>(w, bias, e, i));
  }
#pragma unroll
  for (int i = 0; i < S; ++i) {
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) a = __builtin_fmaf(w[k], dp[i + W - 1 - k], a);
    dx[i] = a;
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k] = __builtin_fmaf(dp[i], e[i + k], dw[k]);
    dw[W] += dp[i];
  }
}

// dfinal's share of the gradient of place m of e (final_state[k] is place len + k).
template <typename Elem, int W>
__device__ __forceinline__ float dfinal_at(const ConvParams& p, int64_t row, uint32_t len, int64_t m) {
  if (!p.dfinal || m < len || m >= int64_t(len) + W - 1) return 0.0f;
  return widen<Elem>(static_cast<const Elem*>(p.dfinal)[row * (W - 1) + (m - len)]);
}

// dfinal's share of dx of the S steps from t0 on.
template <typename Elem, int W>
__device__ __forceinline__ void add_dfinal(const ConvParams& p, int64_t row, uint32_t len, uint32_t t0,
                                           float (&dx)[S]) {
  if (t0 >= len || int64_t(t0) + S + W - 1 <= len) return;
#pragma unroll
  for (int i = 0; i < S; ++i)
    if (t0 + i < len) dx[i] += dfinal_at<Elem, W>(p, row, len, int64_t(t0) + i + W - 1);
}

// The gradient of a row's initial state, from the row's first steps (one lane per row).
template <typename Elem, int W>
__device__ __forceinline__ void store_dinitial(const ConvParams& p, const Elem* xrow, const Elem* grow,
                                               int64_t row, uint32_t len, const float (&w)[W], float bias) {
  float e[2 * (W - 1)], dp[W - 1];
#pragma unroll
  for (int m = 0; m < 2 * (W - 1); ++m)
    e[m] = m < int64_t(len) + W - 1 ? widen<Elem>(place<Elem, W>(p, xrow, row, m)) : 0.0f;
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    dp[i] = uint32_t(i) < len ? widen<Elem>(grow[i]) : 0.0f;
    if (p.silu) dp[i] *= silu_grad_f(window<W>(w, bias, e, i));
  }
#pragma unroll
  for (int m = 0; m < W - 1; ++m) {
    float a = dfinal_at<Elem, W>(p, row, len, m);
#pragma unroll
    for (int k = 0; k <= m; ++k) a = __builtin_fmaf(w[k], dp[m - k], a);
    static_cast<Elem*>(p.dinitial)[row * (W - 1) + m] = narrow<Elem>(a);
  }
}

// Time order: a wave walks kConvBwdTiles tiles of its rows (lanes along time, as the forward).
template <typename Elem, int W>
__global__ __launch_bounds__(kThreads) void conv_bwd_time(ConvParams p) {
  const TimeLane a = time_lane(p);
  const int b = blockIdx.y;
  const int64_t row = int64_t(b) * p.dim + (a.live ? a.d : 0);
  const uint32_t d = a.live ? a.d : 0;
  const uint32_t len = row_length(p, b);
  const Elem* xrow = static_cast<const Elem*>(p.x) + b * p.xb + d * p.xc;
  const Elem* grow = static_cast<const Elem*>(p.dout) + row * p.seqlen;
  Elem* dxrow = static_cast<Elem*>(p.dx) + b * p.dxb + d * p.dxc;
  const uint32_t step = uint32_t(S) << p.lanes_log2, start = a.run * kConvBwdTiles * step + a.j * S;
  float w[W], bias, dw[W + 1];
  load_weights<W>(p, d, w, bias);
#pragma unroll
  for (int k = 0; k <= W; ++k) dw[k] = 0.0f;
  if (a.live) {
    for (int q = 0; q < kConvBwdTiles; ++q) {
      const uint32_t t0 = start + q * step;
      if (t0 >= p.seqlen) break;
      float e[S + 2 * (W - 1)], g[S + W - 1], own[S], next[4], dx[S];
      const int n = steps_left(len, t0);
      load_run<Elem, S>(xrow + t0, n, own);
#pragma unroll
      for (int i = 0; i < S; ++i) e[W - 1 + i] = own[i];
      load_run<Elem, S>(grow + t0, n, own);
#pragma unroll
      for (int i = 0; i < S; ++i) g[i] = own[i];
      load_few<Elem, 4>(xrow + t0 + S, n - S, next);
#pragma unroll
      for (int i = 0; i < W - 1; ++i) e[W - 1 + S + i] = next[i];
      load_few<Elem, 4>(grow + t0 + S, n - S, next);
#pragma unroll
      for (int i = 0; i < W - 1; ++i) g[S + i] = next[i];
      if (t0 == 0)
        load_initial<Elem, W>(p, row, e);
      else
        load_left<Elem, W>(xrow, t0, len, e);
      conv_grad_block<W>(w, bias, p.silu, e, g, dx, dw);
      if (p.dfinal) add_dfinal<Elem, W>(p, row, len, t0, dx);
      store_run_stream<Elem, S>(dxrow + t0, steps_left(p.seqlen, t0), dx);
    }
    if (p.dinitial && a.run == 0 && a.j == 0) store_dinitial<Elem, W>(p, xrow, grow, row, len, w, bias);
  }
  // Sum over the row's lanes, then one store per row.
  for (int m = 1 << p.lanes_log2 >> 1; m > 0; m >>= 1)
#pragma unroll
    for (int k = 0; k <= W; ++k) dw[k] += __shfl_xor(dw[k], m, 64);
  if (a.live && a.j == 0) {
    float* part = p.part + ((int64_t(b) * p.tiles + a.run) * p.dim + d) * (W + 1);
#pragma unroll
    for (int k = 0; k <= W; ++k) part[k] = dw[k];
  }
}

// dx of a lane's channels by S steps, gathered channel by channel into the words of its steps
// (bf16: two channels a dword, when the second has come).
template <typename Elem, int CV>
struct StepWords {
  Word<Elem, CV> w[S];
  float even[S];
  __device__ __forceinline__ void put(int c, const float (&dx)[S]) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if constexpr (sizeof(Elem) == 4) {
        w[i].w[c] = __float_as_uint(dx[i]);
      } else if (c & 1) {
        uint32_t d = pack_bf16x2(even[i], dx[i]);
        asm volatile("" : "+v"(d));  // now, not with the store: half the registers
        w[i].w[c / 2] = d;
      } else {
        even[i] = dx[i];
      }
    }
  }
};

// Channel order: as the forward, dout's words of all channels in flight with x's; the lanes'
// sums meet in LDS.
template <typename Elem, int W>
__global__ __launch_bounds__(kThreads, sizeof(Elem) == 2 ? 4 : 3) void conv_bwd_chan(ConvParams p) {
  constexpr int CV = kConvLaneChannels, K = W + 1;
  using L = ChanLane<CV>;
  constexpr int kRows = kConvWaves * L::TB;  // of sums: a lane along time each
  __shared__ float sw[CW * (W + 1)], sums[kRows][CW * K + 1];
  const L a = chan_lane<CV, true>(p);
  Weights<W> weights;
  weights.load(p, a.cb);
  const int b = a.b;
  const bool live = a.nc > 0 && a.t0 < p.seqlen;
  const uint32_t len = row_length(p, b);
  const int64_t row0 = int64_t(b) * p.dim + a.c0;
  const Elem* xb = static_cast<const Elem*>(p.x) + b * p.xb + a.c0;
  const Elem* gb = static_cast<const Elem*>(p.dout) + row0 * p.seqlen + a.t0;
  const int n = live ? steps_left(len, a.t0) : 0;
  Word<Elem, CV> raw[S + 2 * (W - 1)];
  Word<Elem, S> graw[CV];
  Word<Elem, 4> gnext[CV];
  if (live && len > 0) load_rows<Elem, CV, S + 2 * (W - 1)>(xb, p.xt, int64_t(a.t0) - (W - 1), len, a.nc, raw);
  const bool whole = a.nc >= CV && n >= S + 4;
  // The steps behind a block are the next lane's first where that lies in the wave and is whole.
  const bool last = a.tb == L::TB - 1 || n < 2 * S + 4;
  if (whole) {
#pragma unroll
    for (int c = 0; c < CV; ++c) {
      const Elem* g = gb + int64_t(c) * p.seqlen;
      graw[c] = *reinterpret_cast<const Word<Elem, S>*>(g);
      if (last) gnext[c] = *reinterpret_cast<const Word<Elem, 4>*>(g + S);
    }
  }
  weights.stage(sw);
  const bool first = a.tile == 0 && a.wv == 0;
  if (live && int64_t(a.t0) + S + W - 1 > len) {
#pragma unroll
    for (int i = 0; i < S + 2 * (W - 1); ++i)
      if (int64_t(a.t0) - (W - 1) + i >= len) raw[i] = Word<Elem, CV>{};
  }
#pragma unroll
  for (int c = 0; c < CV; ++c)
#pragma unroll
    for (int q = 0; q < int(sizeof(Elem)); ++q) {
      const uint32_t v = __shfl_down(graw[c].w[q], L::CG, 64);
      gnext[c].w[q] = last ? gnext[c].w[q] : v;
    }
  StepWords<Elem, CV> words;
  float* mine = sums[a.wv * L::TB + a.tb] + a.cl * K;
#pragma unroll
  for (int c = 0; c < CV; ++c) {
    float dw[K];
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k] = 0.0f;
    if (live) {
      float w[W], bias, e[S + 2 * (W - 1)], g[S + W - 1], dx[S];
      Weights<W>::of(sw, a.cl + c, w, bias);
      if (whole) {
#pragma unroll
        for (int i = 0; i < S; ++i) g[i] = few_elem<Elem>(graw[c], i);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) g[S + i] = few_elem<Elem>(gnext[c], i);
      } else {
        load_part_of<Elem, S + W - 1>(gb + int64_t(c) * p.seqlen, c >= a.nc ? 0 : n < S + W - 1 ? n : S + W - 1, g);
      }
#pragma unroll
      for (int i = 0; i < S + 2 * (W - 1); ++i) e[i] = few_elem<Elem>(raw[i], c);
      if (first && a.tb == 0 && c < a.nc) load_initial<Elem, W>(p, row0 + c, e);
      conv_grad_block<W>(w, bias, p.silu, e, g, dx, dw);
      if (p.dfinal && c < a.nc) add_dfinal<Elem, W>(p, row0 + c, len, a.t0, dx);
      words.put(c, dx);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) mine[c * K + k] = dw[k];
  }
  if (live) {
    Elem* dxb = static_cast<Elem*>(p.dx) + b * p.dxb + a.c0 + a.t0 * p.dxt;
    if (a.nc >= CV && a.t0 + S <= p.seqlen) {
#pragma unroll
      for (int i = 0; i < S; ++i) *reinterpret_cast<Word<Elem, CV>*>(dxb + i * p.dxt) = words.w[i];
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        float v[CV];
#pragma unroll
        for (int c = 0; c < CV; ++c) v[c] = few_elem<Elem>(words.w[i], c);
        if (a.t0 + i < p.seqlen) store_few<Elem, CV>(dxb + i * p.dxt, a.nc, v);
      }
    }
    if (p.dinitial && first && a.tb == 0) {
      for (int c = 0; c < CV; ++c) {
        if (c >= a.nc) break;
        float w[W], bias;
        load_weights<W>(p, a.c0 + c, w, bias);
        store_dinitial<Elem, W>(p, xb + c, gb + int64_t(c) * p.seqlen, row0 + c, len, w, bias);
      }
    }
  }
  __syncthreads();
  constexpr int cols = CW * K;
  for (int i = threadIdx.x; i < cols; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) v += sums[r][i];
    const int64_t col = int64_t(a.cb) * cols + i;  // (channel, k)
    if (col < int64_t(p.dim) * K) p.part[(int64_t(b) * p.tiles + a.tile) * p.dim * K + col] = v;
  }
}

struct ReduceParams {
  const float* part;  // [rows][cols]
  float* dweight;     // [dim, W]
  float* dbias;       // nullable
  int64_t rows, cols;
  int width;
};

__global__ __launch_bounds__(kReduceCols* kConvReduceSlices) void conv_bwd_reduce(ReduceParams p) {
  __shared__ float buf[kConvReduceSlices][kReduceCols + 1];
  const int64_t col = int64_t(blockIdx.x) * kReduceCols + threadIdx.x % kReduceCols;
  const float a = sum_rows<kReduceCols, kConvReduceSlices>(p.part, p.rows, p.cols, col, buf);
  if (threadIdx.x >= kReduceCols || col >= p.cols) return;
  const int64_t d = col / (p.width + 1);
  const int k = int(col - d * (p.width + 1));
  if (k < p.width)
    p.dweight[d * p.width + k] = a;
  else if (p.dbias)
    p.dbias[d] = a;
}

ConvParams params_of(const ConvArgs& a) {
  ConvParams p{};
  p.x = a.x;
  p.xb = a.xs.batch;
  p.xc = a.xs.channel;
  p.xt = a.xs.step;
  p.weight = a.weight;
  p.bias = a.bias;
  p.initial = a.initial;
  p.lengths = a.lengths;
  p.out = a.out;
  p.final_state = a.final_state;
  p.dout = a.dout;
  p.dfinal = a.dfinal;
  p.dx = a.dx;
  p.dxb = a.dxs.batch;
  p.dxc = a.dxs.channel;
  p.dxt = a.dxs.step;
  p.dinitial = a.dinitial;
  p.part = a.workspace;
  p.dim = uint32_t(a.dim);
  p.seqlen = uint32_t(a.seqlen);
  p.silu = a.silu ? 1 : 0;
  p.lanes_log2 = conv_row_lanes_log2(a.seqlen);
  return p;
}

dim3 grid_of(const ConvArgs& a, const ConvGrid& g, ConvParams* p) {
  p->tiles = uint32_t(g.tiles);
  p->waves = uint32_t(g.waves);
  return dim3(unsigned(g.groups), unsigned(a.batch));
}

template <typename Elem, int W, int T>
void run_fwd_time(const ConvArgs& a, ConvParams& p, hipStream_t s) {
  const dim3 grid = grid_of(a, conv_time_grid(a.dim, a.seqlen, T), &p);
  hipLaunchKernelGGL((conv_fwd_time<Elem, W, T>), grid, dim3(kThreads), 0, s, p);
}

template <typename Elem, int W>
void run_fwd(const ConvArgs& a, ConvParams& p, hipStream_t s) {
  if (a.order == Order::Time || a.seqlen == 0) {
    if constexpr (sizeof(Elem) == 2) {
      if (conv_fwd_wave_tiles(a.batch, a.dim, a.seqlen, a.io) == 2) return run_fwd_time<Elem, W, 2>(a, p, s);
    }
    run_fwd_time<Elem, W, 1>(a, p, s);
  } else {
    const dim3 grid = grid_of(a, conv_chan_grid(a.dim, a.seqlen), &p);
    hipLaunchKernelGGL((conv_fwd_chan<Elem, W>), grid, dim3(kThreads), 0, s, p);
  }
}

template <typename Elem, int W>
void run_bwd(const ConvArgs& a, ConvParams& p, hipStream_t s) {
  if (a.order == Order::Time || a.seqlen == 0) {
    const dim3 grid = grid_of(a, conv_time_grid(a.dim, a.seqlen, kConvBwdTiles), &p);
    hipLaunchKernelGGL((conv_bwd_time<Elem, W>), grid, dim3(kThreads), 0, s, p);
  } else {
    const dim3 grid = grid_of(a, conv_chan_grid(a.dim, a.seqlen), &p);
    hipLaunchKernelGGL((conv_bwd_chan<Elem, W>), grid, dim3(kThreads), 0, s, p);
  }
}

// f<Elem, W>(...) for the storage type and width.
#define SSM_CONV_DISPATCH(f, ...)                                                         \
  if (a.io == Io::BF16)                                                                   \
    a.width == 2 ? f<uint16_t, 2>(__VA_ARGS__)                                            \
                 : a.width == 3 ? f<uint16_t, 3>(__VA_ARGS__) : f<uint16_t, 4>(__VA_ARGS__); \
  else                                                                                    \
    a.width == 2 ? f<float, 2>(__VA_ARGS__)                                               \
                 : a.width == 3 ? f<float, 3>(__VA_ARGS__) : f<float, 4>(__VA_ARGS__);

}  // namespace

int launch_conv_fwd(const ConvArgs& a, void* stream) {
  ConvParams p = params_of(a);
  hipStream_t s = static_cast<hipStream_t>(stream);
  SSM_CONV_DISPATCH(run_fwd, a, p, s)
  return int(hipGetLastError());
}

int launch_conv_bwd(const ConvArgs& a, void* stream) {
  ConvParams p = params_of(a);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.batch > 0) {
    SSM_CONV_DISPATCH(run_bwd, a, p, s)
    const int err = int(hipGetLastError());
    if (err) return err;
  }
  ReduceParams r{a.workspace, a.dweight, a.dbias, a.batch * int64_t(p.tiles),
                 a.dim * (a.width + 1), int(a.width)};
  hipLaunchKernelGGL(conv_bwd_reduce, dim3(unsigned(reduce_groups(r.cols))), dim3(kReduceCols * kConvReduceSlices),
                     0, s, r);
  return int(hipGetLastError());
}

// ---------------------------------------------------------------- single-token step
//
// A lane holds four bytes of channels (one fp32, two bf16), so that x, the W - 1 past inputs of
// each (W - 1 dwords) and the weights are contiguous over a wave, and takes R rows, whose
// loads are in flight together and share the weights. Rows that name one slot are taken in
// row order by the first of them, so each sees the state the row before it left.

namespace {

struct ConvStepParams {
  const void* x;
  int64_t x_stride;
  void* state;
  const float* weight;
  const float* bias;
  const int32_t* slots;
  void* out;
  int64_t nslots;
  int batch, dim, silu;
};

template <typename Elem, int W, int R>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepParams p) {
  constexpr int CV = 4 / int(sizeof(Elem));
  const int64_t c0 = (int64_t(blockIdx.x) * 256 + threadIdx.x) * CV;
  // Channels of this lane; a lane past the last one keeps its wave's searches whole.
  const int n = c0 >= p.dim ? 0 : p.dim - c0 < CV ? int(p.dim - c0) : CV;
  const int r0 = blockIdx.y * R;
  const Elem* xs = static_cast<const Elem*>(p.x) + c0;
  Elem* out = static_cast<Elem*>(p.out) + c0;
  auto state_of = [&](int slot) { return static_cast<Elem*>(p.state) + (int64_t(slot) * p.dim + c0) * (W - 1); };

  __shared__ int found[2][kConvWaves][2];
  int turn = 0;
  float past[R][CV * (W - 1)], x[R][CV], w[CV * W], bias[CV];
  int slot[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + i;
    slot[i] = r >= p.batch ? -1 : p.slots ? p.slots[r] : r;
    if (slot[i] >= p.nslots) slot[i] = -1;
    load_few<Elem, CV>(xs + r * p.x_stride, r < p.batch ? n : 0, x[i]);
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    load_few<Elem, CV*(W - 1)>(state_of(slot[i]), slot[i] >= 0 ? n * (W - 1) : 0, past[i]);
  load_few<float, CV * W>(p.weight + c0 * W, n * W, w);
  load_few<float, CV>(p.bias + c0, p.bias ? n : 0, bias);
  SlotOrder order[R];
#pragma unroll
  for (int i = 0; i < R; ++i) order[i] = SlotOrder{true, INT32_MAX};
  if (p.slots) slot_order<kConvWaves, R>(p.slots, p.batch, r0, slot, found, turn, order);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    int r = r0 + i;
    if (r >= p.batch) break;
    // (a row of no slot is its own; else the first row of a slot takes the later ones)
    if (slot[i] >= 0 && !order[i].first) continue;
    for (;;) {
      float o[CV];
#pragma unroll
      for (int c = 0; c < CV; ++c) {
        float acc = bias[c];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) acc = __builtin_fmaf(w[c * W + k], past[i][c * (W - 1) + k], acc);
        acc = __builtin_fmaf(w[c * W + W - 1], x[i][c], acc);
        if (p.silu) acc = silu_f(acc);
        o[c] = slot[i] >= 0 ? acc : 0.0f;  // a row of no slot: zeros
#pragma unroll
        for (int k = 0; k < W - 2; ++k) past[i][c * (W - 1) + k] = past[i][c * (W - 1) + k + 1];
        past[i][c * (W - 1) + W - 2] = x[i][c];
      }
      store_few<Elem, CV>(out + int64_t(r) * p.dim, n, o);
      if (slot[i] < 0 || order[i].next == INT32_MAX) break;
      r = order[i].next;
      SlotOrder following[1];
      const int one[1] = {slot[i]};
      slot_order<kConvWaves, 1>(p.slots, p.batch, r, one, found, turn ^= 1, following);
      order[i].next = following[0].next;
      load_few<Elem, CV>(xs + r * p.x_stride, n, x[i]);
    }
    if (slot[i] >= 0) store_few<Elem, CV*(W - 1)>(state_of(slot[i]), n * (W - 1), past[i]);
  }
}

template <typename Elem, int W, int R>
void run_step_rows(const ConvStepArgs& a, const ConvStepParams& p, hipStream_t s) {
  constexpr int per = 256 * 4 / int(sizeof(Elem));
  const dim3 grid(unsigned((a.dim + per - 1) / per), unsigned((a.batch + R - 1) / R));
  hipLaunchKernelGGL((conv_step_kernel<Elem, W, R>), grid, dim3(256), 0, s, p);
}

template <typename Elem, int W>
void run_step(const ConvStepArgs& a, const ConvStepParams& p, hipStream_t s) {
  if (conv_step_rows(a.batch, a.dim, a.io) == 2)
    run_step_rows<Elem, W, 2>(a, p, s);
  else
    run_step_rows<Elem, W, 1>(a, p, s);
}

}  // namespace

int launch_conv_step(const ConvStepArgs& a, void* stream) {
  ConvStepParams p{a.x, a.x_stride, a.state, a.weight, a.bias, a.slots, a.out, a.nslots,
                   int(a.batch), int(a.dim), a.silu ? 1 : 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  SSM_CONV_DISPATCH(run_step, a, p, s)
  return int(hipGetLastError());
}

}  // namespace ssm
