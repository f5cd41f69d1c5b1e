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
//   channel  runs of channels (a slice of a projection's output): a lane holds 16 bytes of
//            channels by 8 steps, loads one 16-byte word per step and stores one run of
//            steps per channel, which turns the order through registers alone. A wave
//            covers 64 channels by 64 (bf16) or 32 (fp32) steps: 128-byte or longer
//            segments on both sides.
// Sums are fp32; a result is rounded once, at its store. A row's steps at and behind its
// length are never read; its outputs there are zeros.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_launch.h"
#include "device_block.h"

namespace ssm {
namespace {

constexpr int S = kConvSteps;
constexpr int kThreads = 64 * kConvWaves;

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
  int batch, dim, seqlen;
  int silu;
  uint32_t waves;    // time order: waves with work
  uint32_t tiles;    // runs of steps per row
  int lanes_log2;    // time order: lanes along a row
  uint32_t cblocks;  // channel order: blocks of 64 channels
};

__device__ __forceinline__ int row_length(const ConvParams& p, int b) {
  if (!p.lengths) return p.seqlen;
  const int n = p.lengths[b];
  return n < 0 ? 0 : n > p.seqlen ? p.seqlen : n;
}

template <int W>
__device__ __forceinline__ void load_weights(const ConvParams& p, int d, float (&w)[W], float& bias) {
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = p.weight[int64_t(d) * W + k];
  bias = p.bias ? p.bias[d] : 0.0f;
}

// Place m of e: the initial state for m < W - 1 (zero without one), x at step m - (W - 1).
template <typename Elem, int W>
__device__ __forceinline__ Elem place(const ConvParams& p, const Elem* xrow, int b, int d, int64_t m) {
  if (m >= W - 1) return xrow[(m - (W - 1)) * p.xt];
  if (!p.initial) return Elem(0);
  return static_cast<const Elem*>(p.initial)[(int64_t(b) * p.dim + d) * (W - 1) + m];
}

// The last W - 1 inputs before the row's end (one lane per row).
template <typename Elem, int W>
__device__ __forceinline__ void store_final(const ConvParams& p, const Elem* xrow, int b, int d, int len) {
  Elem* f = static_cast<Elem*>(p.final_state) + (int64_t(b) * p.dim + d) * (W - 1);
#pragma unroll
  for (int k = 0; k < W - 1; ++k) f[k] = place<Elem, W>(p, xrow, b, d, int64_t(len) + k);
}

// e[i] = the input of step t0 - (W - 1) + i, i < W - 1, from memory (a block's left edge).
template <typename Elem, int W, int E>
__device__ __forceinline__ void load_left(const ConvParams& p, const Elem* xrow, int b, int d, int t0,
                                          int len, float (&e)[E]) {
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    const int64_t m = int64_t(t0) + i;
    e[i] = m < int64_t(len) + W - 1 ? widen<Elem>(place<Elem, W>(p, xrow, b, d, m)) : 0.0f;
  }
}

template <int W, int E>
__device__ __forceinline__ float window(const float (&w)[W], float bias, const float (&e)[E], int i) {
  float acc = bias;
#pragma unroll
  for (int k = 0; k < W; ++k) acc = __builtin_fmaf(w[k], e[i + k], acc);
  return acc;
}

// ---------------------------------------------------------------- forward, time order

template <typename Elem, int W>
__global__ __launch_bounds__(kThreads) void conv_fwd_time(ConvParams p) {
  const int lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * kConvWaves + (threadIdx.x >> 6);
  if (wave >= p.waves) return;
  const uint32_t group = wave / p.tiles, tile = wave - group * p.tiles;
  const int lanes = 1 << p.lanes_log2;
  const int j = lane & (lanes - 1);
  const int64_t row = (int64_t(group) << (6 - p.lanes_log2)) + (lane >> p.lanes_log2);
  if (row >= int64_t(p.batch) * p.dim) return;
  const int b = int(uint32_t(row) / uint32_t(p.dim)), d = int(row - int64_t(b) * p.dim);
  const int len = row_length(p, b);
  const Elem* xrow = static_cast<const Elem*>(p.x) + b * p.xb + d * p.xc;
  const int64_t t0 = (int64_t(tile) * lanes + j) * S;
  float w[W], bias, e[S + W - 1], own[S];
  load_weights<W>(p, d, w, bias);
  load_run<Elem, S>(xrow + t0, t0 < len ? int(len - t0) : 0, own);
#pragma unroll
  for (int i = 0; i < S; ++i) e[W - 1 + i] = own[i];
  // The left edge is the last steps of the lane before (of the same row, so active too).
#pragma unroll
  for (int i = 0; i < W - 1; ++i) e[i] = shift_up_one(own[S - (W - 1) + i], 0.0f);
  if (j == 0 && t0 < p.seqlen) load_left<Elem, W>(p, xrow, b, d, int(t0), len, e);
  if (t0 < p.seqlen) {
    float o[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float v = window<W>(w, bias, e, i);
      if (p.silu) v = silu_f(v);
      o[i] = t0 + i < len ? v : 0.0f;
    }
    Elem* orow = static_cast<Elem*>(p.out) + row * p.seqlen;
    store_run<Elem, S>(orow + t0, int(p.seqlen - t0 < S ? p.seqlen - t0 : S), o);
  }
  if (p.final_state && tile == 0 && j == 0) store_final<Elem, W>(p, xrow, b, d, len);
}

// ---------------------------------------------------------------- forward, channel order

template <typename Elem, int W>
__global__ __launch_bounds__(kThreads) void conv_fwd_chan(ConvParams p) {
  constexpr int CV = Vec<Elem>::kN;        // channels per lane
  constexpr int CG = 64 / CV;              // lanes along channels: 64 channels
  constexpr int TB = 64 / CG;              // lanes along time
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const uint32_t tile = blockIdx.x % p.tiles, rest = blockIdx.x / p.tiles;
  const uint32_t cb = rest % p.cblocks;
  const int b = int(rest / p.cblocks);
  const int c0 = int(cb) * 64 + (lane % CG) * CV;
  const int64_t t0 = ((int64_t(tile) * kConvWaves + wv) * TB + lane / CG) * S;
  const int nc = p.dim - c0;  // channels from c0 on
  if (nc <= 0 || t0 >= p.seqlen) return;
  const int len = row_length(p, b);
  const Elem* xb = static_cast<const Elem*>(p.x) + b * p.xb + c0;
  uint4 raw[S + W - 1];
#pragma unroll
  for (int i = 0; i < S + W - 1; ++i) {
    const int64_t t = t0 - (W - 1) + i;
    raw[i] = t >= 0 && t < len ? load_word_n<Elem>(xb + t * p.xt, nc) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int c = 0; c < CV; ++c) {
    if (c >= nc) break;
    const int d = c0 + c;
    float w[W], bias, e[S + W - 1], o[S];
    load_weights<W>(p, d, w, bias);
#pragma unroll
    for (int i = 0; i < S + W - 1; ++i) e[i] = word_elem<Elem>(raw[i], c);
    if (t0 == 0) load_left<Elem, W>(p, xb + c, b, d, 0, len, e);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      float v = window<W>(w, bias, e, i);
      if (p.silu) v = silu_f(v);
      o[i] = t0 + i < len ? v : 0.0f;
    }
    Elem* orow = static_cast<Elem*>(p.out) + (int64_t(b) * p.dim + d) * p.seqlen;
    store_run<Elem, S>(orow + t0, int(p.seqlen - t0 < S ? p.seqlen - t0 : S), o);
    if (p.final_state && t0 == 0) store_final<Elem, W>(p, xb + c, b, d, len);
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
  for (int i = 0; i < S + W - 1; ++i)
    dp[i] = silu ? g[i] * silu_grad_f(window<W>(w, bias, e, i)) : g[i];
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
__device__ __forceinline__ float dfinal_at(const ConvParams& p, int64_t row, int len, int64_t m) {
  if (!p.dfinal || m < len || m >= int64_t(len) + W - 1) return 0.0f;
  return widen<Elem>(static_cast<const Elem*>(p.dfinal)[row * (W - 1) + (m - len)]);
}

template <typename Elem, int W>
__device__ __forceinline__ void store_dinitial(const ConvParams& p, int64_t row, int len, const float (&w)[W],
                                               const float (&dp)[W - 1]) {
#pragma unroll
  for (int m = 0; m < W - 1; ++m) {
    float a = dfinal_at<Elem, W>(p, row, len, m);
#pragma unroll
    for (int k = 0; k <= m; ++k) a = __builtin_fmaf(w[k], dp[m - k], a);
    static_cast<Elem*>(p.dinitial)[row * (W - 1) + m] = narrow<Elem>(a);
  }
}

// dp of the first W - 1 steps, for dinitial.
template <int W>
__device__ __forceinline__ void first_dp(const float (&w)[W], float bias, bool silu,
                                         const float (&e)[S + 2 * (W - 1)],
                                         const float (&g)[S + W - 1], float (&dp)[W - 1]) {
#pragma unroll
  for (int i = 0; i < W - 1; ++i)
    dp[i] = silu ? g[i] * silu_grad_f(window<W>(w, bias, e, i)) : g[i];
}

// Time order: a wave walks kConvBwdTiles tiles of its rows (lanes along time, as the forward).
template <typename Elem, int W>
__global__ __launch_bounds__(kThreads) void conv_bwd_time(ConvParams p) {
  const int lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * kConvWaves + (threadIdx.x >> 6);
  if (wave >= p.waves) return;
  const uint32_t group = wave / p.tiles, run = wave - group * p.tiles;
  const int lanes = 1 << p.lanes_log2;
  const int j = lane & (lanes - 1);
  const int64_t row = (int64_t(group) << (6 - p.lanes_log2)) + (lane >> p.lanes_log2);
  const bool live = row < int64_t(p.batch) * p.dim;
  const int b = live ? int(uint32_t(row) / uint32_t(p.dim)) : 0;
  const int d = live ? int(row - int64_t(b) * p.dim) : 0;
  const int len = live ? row_length(p, b) : 0;
  const Elem* xrow = static_cast<const Elem*>(p.x) + b * p.xb + d * p.xc;
  const Elem* grow = static_cast<const Elem*>(p.dout) + (live ? row : 0) * p.seqlen;
  Elem* dxrow = static_cast<Elem*>(p.dx) + b * p.dxb + d * p.dxc;
  float w[W], bias, dw[W + 1];
  load_weights<W>(p, d, w, bias);
#pragma unroll
  for (int k = 0; k <= W; ++k) dw[k] = 0.0f;
  for (int q = 0; q < kConvBwdTiles; ++q) {
    const int64_t t0 = ((int64_t(run) * kConvBwdTiles + q) * lanes + j) * S;
    if (!live || (t0 >= p.seqlen && t0 > 0)) break;  // (an empty row still has its states)
    float e[S + 2 * (W - 1)], g[S + W - 1], own[S], dx[S];
    const int n = t0 < len ? int(len - t0 < 2 * S ? len - t0 : 2 * S) : 0;  // steps from t0 on
    load_run<Elem, S>(xrow + t0, n, own);
#pragma unroll
    for (int i = 0; i < S; ++i) e[W - 1 + i] = own[i];
    load_left<Elem, W>(p, xrow, b, d, int(t0), len, e);
    load_run<Elem, S>(grow + t0, n, own);
#pragma unroll
    for (int i = 0; i < S; ++i) g[i] = own[i];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
      e[W - 1 + S + i] = S + i < n ? widen<Elem>(xrow[t0 + S + i]) : 0.0f;
      g[S + i] = S + i < n ? widen<Elem>(grow[t0 + S + i]) : 0.0f;
    }
    conv_grad_block<W>(w, bias, p.silu, e, g, dx, dw);
    if (t0 == 0 && p.dinitial) {
      float dp[W - 1];
      first_dp<W>(w, bias, p.silu, e, g, dp);
      store_dinitial<Elem, W>(p, row, len, w, dp);
    }
    if (p.dfinal && t0 + S + W - 1 > len && t0 < len) {
#pragma unroll
      for (int i = 0; i < S; ++i)
        if (t0 + i < len) dx[i] += dfinal_at<Elem, W>(p, row, len, t0 + i + W - 1);
    }
    store_run<Elem, S>(dxrow + t0, int(p.seqlen - t0 < S ? p.seqlen - t0 : S), dx);
  }
  // Sum over the row's lanes, then one store per row.
  for (int m = lanes >> 1; m > 0; m >>= 1)
#pragma unroll
    for (int k = 0; k <= W; ++k) dw[k] += __shfl_xor(dw[k], m, 64);
  if (live && j == 0) {
    float* part = p.part + ((int64_t(b) * p.tiles + run) * p.dim + d) * (W + 1);
#pragma unroll
    for (int k = 0; k <= W; ++k) part[k] = dw[k];
  }
}

// Channel order: as the forward; the lanes' sums meet in LDS.
template <typename Elem, int W>
__global__ __launch_bounds__(kThreads) void conv_bwd_chan(ConvParams p) {
  constexpr int CV = Vec<Elem>::kN;
  constexpr int CG = 64 / CV;
  constexpr int TB = 64 / CG;
  constexpr int K = W + 1;
  __shared__ float sums[kConvWaves * TB][64 * K + 1];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const uint32_t tile = blockIdx.x % p.tiles, rest = blockIdx.x / p.tiles;
  const uint32_t cb = rest % p.cblocks;
  const int b = int(rest / p.cblocks);
  const int cl = (lane % CG) * CV;
  const int c0 = int(cb) * 64 + cl;
  const int64_t t0 = ((int64_t(tile) * kConvWaves + wv) * TB + lane / CG) * S;
  const int nc = p.dim - c0;
  const int len = row_length(p, b);
  float* mine = sums[wv * TB + lane / CG] + cl * K;
  if (nc > 0 && t0 < p.seqlen) {
    const Elem* xb = static_cast<const Elem*>(p.x) + b * p.xb + c0;
    uint4 raw[S + 2 * (W - 1)];
    float dxw[S][CV];
#pragma unroll
    for (int i = 0; i < S + 2 * (W - 1); ++i) {
      const int64_t t = t0 - (W - 1) + i;
      raw[i] = t >= 0 && t < len ? load_word_n<Elem>(xb + t * p.xt, nc) : make_uint4(0, 0, 0, 0);
    }
    const int n = t0 < len ? int(len - t0 < 2 * S ? len - t0 : 2 * S) : 0;
#pragma unroll
    for (int c = 0; c < CV; ++c) {
      float dw[K];
#pragma unroll
      for (int k = 0; k < K; ++k) dw[k] = 0.0f;
      if (c < nc) {
        const int d = c0 + c;
        const int64_t row = int64_t(b) * p.dim + d;
        const Elem* grow = static_cast<const Elem*>(p.dout) + row * p.seqlen;
        float w[W], bias, e[S + 2 * (W - 1)], g[S + W - 1], own[S], dx[S];
        load_weights<W>(p, d, w, bias);
        load_run<Elem, S>(grow + t0, n, own);
#pragma unroll
        for (int i = 0; i < S; ++i) g[i] = own[i];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) g[S + i] = S + i < n ? widen<Elem>(grow[t0 + S + i]) : 0.0f;
#pragma unroll
        for (int i = 0; i < S + 2 * (W - 1); ++i) e[i] = word_elem<Elem>(raw[i], c);
        if (t0 == 0) load_left<Elem, W>(p, xb + c, b, d, 0, len, e);
        conv_grad_block<W>(w, bias, p.silu, e, g, dx, dw);
        if (t0 == 0 && p.dinitial) {
          float dp[W - 1];
          first_dp<W>(w, bias, p.silu, e, g, dp);
          store_dinitial<Elem, W>(p, row, len, w, dp);
        }
        if (p.dfinal && t0 + S + W - 1 > len && t0 < len) {
#pragma unroll
          for (int i = 0; i < S; ++i)
            if (t0 + i < len) dx[i] += dfinal_at<Elem, W>(p, row, len, t0 + i + W - 1);
        }
#pragma unroll
        for (int i = 0; i < S; ++i) dxw[i][c] = dx[i];
      } else {
#pragma unroll
        for (int i = 0; i < S; ++i) dxw[i][c] = 0.0f;
      }
#pragma unroll
      for (int k = 0; k < K; ++k) mine[c * K + k] = dw[k];
    }
    Elem* dxb = static_cast<Elem*>(p.dx) + b * p.dxb + c0;
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (t0 + i < p.seqlen) store_run<Elem, CV>(dxb + (t0 + i) * p.dxt, nc < CV ? nc : CV, dxw[i]);
  } else {
#pragma unroll
    for (int i = 0; i < CV * K; ++i) mine[i] = 0.0f;
  }
  __syncthreads();
  const int cols = 64 * K;
  for (int i = threadIdx.x; i < cols; i += kThreads) {
    float a = 0.0f;
#pragma unroll
    for (int r = 0; r < kConvWaves * TB; ++r) a += sums[r][i];
    const int64_t col = int64_t(cb) * cols + i;  // (channel, k)
    if (col < int64_t(p.dim) * K)
      p.part[(int64_t(b) * p.tiles + tile) * p.dim * K + col] = a;
  }
}

struct ReduceParams {
  const float* part;  // [rows][cols]
  float* dweight;     // [dim, W]
  float* dbias;       // nullable
  int64_t rows, cols;
  int width;
};

constexpr int kReduceCols = 32, kReduceSlices = 16;

__global__ __launch_bounds__(kReduceCols* kReduceSlices) void conv_bwd_reduce(ReduceParams p) {
  __shared__ float buf[kReduceSlices][kReduceCols + 1];
  const int64_t col = int64_t(blockIdx.x) * kReduceCols + threadIdx.x % kReduceCols;
  const float a = sum_rows<kReduceCols, kReduceSlices>(p.part, p.rows, p.cols, col, buf);
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
  p.batch = int(a.batch);
  p.dim = int(a.dim);
  p.seqlen = int(a.seqlen);
  p.silu = a.silu ? 1 : 0;
  p.lanes_log2 = conv_row_lanes_log2(a.seqlen);
  p.cblocks = uint32_t((a.dim + 63) / 64);
  return p;
}

// Workgroups of the time-ordered kernels, `run` steps of a row per wave.
unsigned time_grid(const ConvArgs& a, ConvParams* p, int64_t run) {
  const int64_t rows = a.batch * a.dim, per = int64_t(1) << (6 - p->lanes_log2);
  p->tiles = a.seqlen > 0 ? uint32_t((a.seqlen + run - 1) / run) : 1;
  p->waves = uint32_t((rows + per - 1) / per * p->tiles);
  return (p->waves + kConvWaves - 1) / kConvWaves;
}

unsigned chan_grid(const ConvArgs& a, ConvParams* p) {
  const int64_t run = conv_channel_tile_steps(a.io);
  p->tiles = uint32_t((a.seqlen + run - 1) / run);
  return unsigned(p->tiles) * p->cblocks * unsigned(a.batch);
}

template <typename Elem, int W>
void run_fwd(const ConvArgs& a, ConvParams& p, hipStream_t s) {
  if (a.order == Order::Time || a.seqlen == 0) {
    const unsigned grid = time_grid(a, &p, int64_t(S) << p.lanes_log2);
    hipLaunchKernelGGL((conv_fwd_time<Elem, W>), dim3(grid), dim3(kThreads), 0, s, p);
  } else {
    const unsigned grid = chan_grid(a, &p);
    hipLaunchKernelGGL((conv_fwd_chan<Elem, W>), dim3(grid), dim3(kThreads), 0, s, p);
  }
}

template <typename Elem, int W>
void run_bwd(const ConvArgs& a, ConvParams& p, hipStream_t s) {
  if (a.order == Order::Time || a.seqlen == 0) {
    const unsigned grid = time_grid(a, &p, (int64_t(S) << p.lanes_log2) * kConvBwdTiles);
    hipLaunchKernelGGL((conv_bwd_time<Elem, W>), dim3(grid), dim3(kThreads), 0, s, p);
  } else {
    const unsigned grid = chan_grid(a, &p);
    hipLaunchKernelGGL((conv_bwd_chan<Elem, W>), dim3(grid), dim3(kThreads), 0, s, p);
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
  const unsigned grid = unsigned((r.cols + kReduceCols - 1) / kReduceCols);
  hipLaunchKernelGGL(conv_bwd_reduce, dim3(grid), dim3(kReduceCols * kReduceSlices), 0, s, r);
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

// N dwords at element alignment.
template <int N>
struct __attribute__((packed, aligned(2))) Dwords {
  uint32_t w[N];
};

// The n (of C) values from p on, the rest zero.
template <typename Elem, int C>
__device__ __forceinline__ void load_few(const Elem* p, int n, float (&v)[C]) {
  constexpr int N = C * int(sizeof(Elem)) / 4;
  if (n >= C) {
    const Dwords<N> d = *reinterpret_cast<const Dwords<N>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(Elem) == 4) {
        v[i] = __uint_as_float(d.w[i]);
      } else {
        v[2 * i] = bf16_lo(d.w[i]);
        v[2 * i + 1] = bf16_hi(d.w[i]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = i < n ? widen<Elem>(p[i]) : 0.0f;
  }
}

template <typename Elem, int C>
__device__ __forceinline__ void store_few(Elem* p, int n, const float (&v)[C]) {
  constexpr int N = C * int(sizeof(Elem)) / 4;
  if (n >= C) {
    Dwords<N> d;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (sizeof(Elem) == 4)
        d.w[i] = __float_as_uint(v[i]);
      else
        d.w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
    *reinterpret_cast<Dwords<N>*>(p) = d;
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < n) p[i] = narrow<Elem>(v[i]);
  }
}

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

// Two rows per lane once the rows fill the device's 8192 wave slots, one before that. 384 rows
// of 4352 bf16 channels: 9.6 us with one row, 8.8 with two, 10.2 with four; 8 rows of 2304:
// 2.9 us with one.
template <typename Elem, int W>
void run_step(const ConvStepArgs& a, const ConvStepParams& p, hipStream_t s) {
  const int64_t waves = (a.dim * int64_t(sizeof(Elem)) / 256 + 1) * a.batch;
  if (waves > 8192)
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
