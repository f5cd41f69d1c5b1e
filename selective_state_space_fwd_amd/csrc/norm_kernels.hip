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
// channels contiguous (single tokens) a lane holds one step.
//
// All of it is bound by memory: 3 reads and writes per element forward, 5 backward.
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
  float eps, inv_g;
  int batch, groups, g, seqlen;
  int lanes_log2, blocks, norm_first;
  uint32_t tiles, total;
};

// The words of a lane's square, one per channel (steps within) when kSteps > 1; one word of
// channels when kSteps is 1.
template <typename Elem, int kSteps>
struct Square {
  static constexpr int CV = Vec<Elem>::kN;
  static constexpr int kWords = kSteps > 1 ? CV : 1;
  uint4 w[kWords];
  __device__ __forceinline__ float at(int c, int t) const {
    return kSteps > 1 ? word_elem<Elem>(w[kSteps > 1 ? c : 0], t) : word_elem<Elem>(w[0], c);
  }
};

// Makes the compiler take the words as new: what was computed from them before (the gate's
// exponentials, 64 values a lane) is then formed again after the reduction instead of held
// across it, where it does not fit the registers.
__device__ __forceinline__ void forget_word(uint4& w) {
  asm volatile("" : "+v"(w.x), "+v"(w.y), "+v"(w.z), "+v"(w.w));
}
template <typename Elem, int kSteps>
__device__ __forceinline__ void forget(Square<Elem, kSteps>& s) {
#pragma unroll
  for (int i = 0; i < Square<Elem, kSteps>::kWords; ++i) forget_word(s.w[i]);
}

// Rows and columns of the words exchanged.
template <typename Elem>
__device__ __forceinline__ void turn(uint4 (&w)[Vec<Elem>::kN]);
template <>
__device__ __forceinline__ void turn<float>(uint4 (&w)[4]) {
  const uint4 a = w[0], b = w[1], c = w[2], d = w[3];
  w[0] = make_uint4(a.x, b.x, c.x, d.x);
  w[1] = make_uint4(a.y, b.y, c.y, d.y);
  w[2] = make_uint4(a.z, b.z, c.z, d.z);
  w[3] = make_uint4(a.w, b.w, c.w, d.w);
}
template <>
__device__ __forceinline__ void turn<uint16_t>(uint4 (&w)[8]) {
  uint32_t in[8][4], out[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    in[i][0] = w[i].x;
    in[i][1] = w[i].y;
    in[i][2] = w[i].z;
    in[i][3] = w[i].w;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q)  // halves c of words 2q and 2q + 1
      out[c][q] = __builtin_amdgcn_perm(in[2 * q + 1][c / 2], in[2 * q][c / 2],
                                        (c & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = make_uint4(out[i][0], out[i][1], out[i][2], out[i][3]);
}

// The square at (b, channel c0, step t0): nc channels and nt steps of it exist (<= 0: none).
// Whole squares take straight-line 16-byte loads; the others go word by word.
template <typename Elem, int kSteps>
__device__ __forceinline__ void load_square(const Tensor& x, int b, int64_t c0, int64_t t0, int nc, int nt,
                                            Square<Elem, kSteps>& s) {
  constexpr int CV = Vec<Elem>::kN;
  const Elem* p = static_cast<const Elem*>(x.p) + b * x.b + c0 * x.c + t0 * x.t;
  if constexpr (kSteps == 1) {
    s.w[0] = nt > 0 ? load_word_n<Elem>(p, nc) : make_uint4(0, 0, 0, 0);
  } else {
    const int64_t pitch = x.chan ? x.t : x.c;  // from word to word
    if (nc == CV && nt == kSteps) {
#pragma unroll
      for (int i = 0; i < CV; ++i) s.w[i] = load16_any(p + i * pitch);
    } else {
      const int words = x.chan ? nt : nc, n = x.chan ? nc : nt;
#pragma unroll
      for (int i = 0; i < CV; ++i)
        s.w[i] = i < words ? load_word_n<Elem>(p + i * pitch, n) : make_uint4(0, 0, 0, 0);
    }
    if (x.chan) turn<Elem>(s.w);
  }
}

template <typename Elem, int kSteps>
__device__ __forceinline__ void store_square(const Tensor& x, int b, int64_t c0, int64_t t0, int nc, int nt,
                                             Square<Elem, kSteps>& s) {
  constexpr int CV = Vec<Elem>::kN;
  Elem* p = static_cast<Elem*>(const_cast<void*>(x.p)) + b * x.b + c0 * x.c + t0 * x.t;
  if constexpr (kSteps == 1) {
    if (nt > 0) store_word_n<Elem>(p, nc, s.w[0]);
  } else {
    if (x.chan) turn<Elem>(s.w);
    const int64_t pitch = x.chan ? x.t : x.c;
    if (nc == CV && nt == kSteps) {
#pragma unroll
      for (int i = 0; i < CV; ++i) store16_any(p + i * pitch, s.w[i]);
    } else {
      const int words = x.chan ? nt : nc, n = x.chan ? nc : nt;
#pragma unroll
      for (int i = 0; i < CV; ++i)
        if (i < words) store_word_n<Elem>(p + i * pitch, n, s.w[i]);
    }
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
    s.w[c] = narrow_raw16<Elem>(v);
  } else {
    row[c] = v[0];
    if (c == CV - 1) s.w[0] = narrow_raw16<Elem>(row);
  }
}

// Without a gate, gate first, norm first.
enum Mode { kNoGate = 0, kGateFirst = 1, kNormFirst = 2 };

// Each v[t] summed over the 2^lg consecutive lanes that share its step.
template <int N>
__device__ __forceinline__ void sum_channels(float (&v)[N], int lg) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (lg >= 1) v[i] = dpp_add<0xB1>(v[i]);
    if (lg >= 2) v[i] = dpp_add<0x4E>(v[i]);
    if (lg >= 3) v[i] = dpp_add<0x141>(v[i]);
    if (lg >= 4) v[i] = dpp_add<0x140>(v[i]);
    if (lg >= 5) v[i] += __shfl_xor(v[i], 16, 64);
    if (lg >= 6) v[i] += __shfl_xor(v[i], 32, 64);
  }
}

// ... and over the workgroup's waves, in wave order: buf holds waves x lanes-along-time x N.
template <int N>
__device__ __forceinline__ void sum_group(float (&v)[N], int lg, float* buf) {
  sum_channels<N>(v, lg);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tb = lane >> lg, times = 64 >> lg;
  if ((lane & ((1 << lg) - 1)) == 0) {
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
  int b, grp, tile, nt;
  int64_t t0, c0;  // first step; first channel within the group, of round 0
};

template <typename Elem, int kSteps>
__device__ __forceinline__ Place place_of(const NormParams& p) {
  constexpr int CV = Vec<Elem>::kN;
  const uint32_t id = xcd_order(blockIdx.x, p.total);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Place a;
  a.tile = int(id % p.tiles);
  const uint32_t rest = id / p.tiles;
  a.grp = int(rest % uint32_t(p.groups));
  a.b = int(rest / uint32_t(p.groups));
  a.t0 = (int64_t(a.tile) * (64 >> p.lanes_log2) + (lane >> p.lanes_log2)) * kSteps;
  a.nt = a.t0 >= p.seqlen ? 0 : p.seqlen - a.t0 < kSteps ? int(p.seqlen - a.t0) : kSteps;
  a.c0 = ((int64_t(wave) << p.lanes_log2) + (lane & ((1 << p.lanes_log2) - 1))) * CV;
  return a;
}

template <int CV>
__device__ __forceinline__ int channels_left(const NormParams& p, int64_t c0) {
  return c0 >= p.g ? 0 : p.g - c0 < CV ? int(p.g - c0) : CV;
}

// ---------------------------------------------------------------- forward
//
// kHeld: the group is covered in one round and stays in registers; else the rounds are read a
// second time (groups of more than 16 waves of channels).
template <typename Elem, int kSteps, bool kHeld, int kMode>
__global__ __launch_bounds__(64 * kNormFwdWaves) void norm_fwd_kernel(NormParams p) {
  constexpr int CV = Vec<Elem>::kN;
  extern __shared__ float buf[];
  const Place a = place_of<Elem, kSteps>(p);
  const int64_t round = int64_t(blockDim.x >> 6) * (int64_t(CV) << p.lanes_log2);
  const int64_t base = int64_t(a.grp) * p.g;
  Square<Elem, kSteps> y, z;
  float sum[kSteps];
#pragma unroll
  for (int t = 0; t < kSteps; ++t) sum[t] = 0.0f;
  auto read = [&](int64_t c0) {
    const int nc = channels_left<CV>(p, c0);
    load_square<Elem, kSteps>(p.y, a.b, base + c0, a.t0, nc, a.nt, y);
    if constexpr (kMode != kNoGate) load_square<Elem, kSteps>(p.z, a.b, base + c0, a.t0, nc, a.nt, z);
  };
  auto add = [&]() {
#pragma unroll
    for (int c = 0; c < CV; ++c)
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        float v = y.at(c, t);
        if constexpr (kMode == kGateFirst) v *= silu_f(z.at(c, t));
        sum[t] = __builtin_fmaf(v, v, sum[t]);
      }
  };
  if constexpr (kHeld) {
    read(a.c0);
    add();
  } else {
    for (int k = 0; k < p.blocks; ++k) {
      read(a.c0 + k * round);
      add();
    }
  }
  sum_group<kSteps>(sum, p.lanes_log2, buf);
  float r[kSteps];
#pragma unroll
  for (int t = 0; t < kSteps; ++t) r[t] = __builtin_amdgcn_rsqf(__builtin_fmaf(sum[t], p.inv_g, p.eps));
  if (p.rstd && a.c0 == 0) {
#pragma unroll
    for (int t = 0; t < kSteps; ++t)
      if (t < a.nt) p.rstd[a.b * p.rb + a.grp * p.rg + (a.t0 + t) * p.rt] = r[t];
  }
  auto write = [&](int64_t c0) {
    const int nc = channels_left<CV>(p, c0);
    float w[CV], row[CV];
    load_run<float, CV>(p.weight + base + c0, nc, w);
    Square<Elem, kSteps> o;
#pragma unroll
    for (int c = 0; c < CV; ++c) {
      float v[kSteps];
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        v[t] = y.at(c, t) * (r[t] * w[c]);
        if constexpr (kMode != kNoGate) v[t] *= silu_f(z.at(c, t));
      }
      put<Elem, kSteps>(o, c, v, row);
    }
    store_square<Elem, kSteps>(p.out, a.b, base + c0, a.t0, nc, a.nt, o);
  };
  if constexpr (kHeld) {
    if constexpr (kSteps > 1) {
      forget<Elem, kSteps>(y);
      if constexpr (kMode != kNoGate) forget<Elem, kSteps>(z);
    }
    write(a.c0);
  } else {
    for (int k = 0; k < p.blocks; ++k) {
      read(a.c0 + k * round);
      write(a.c0 + k * round);
    }
  }
}

// ---------------------------------------------------------------- backward
//
// gate first: A = w dout;    S = sum_G A v; dv = r (A - v r^2 S / G); dy = dv s; dz = dv y s'
// norm first: A = w dout s;  S = sum_G A y; dy = r (A - y r^2 S / G); dz = w dout y r s'
// dweight = sum over tokens of dout (s) times the normed value; per workgroup and channel
// here, over workgroups by a second launch in a fixed order.
template <typename Elem, int kSteps, bool kHeld, int kMode>
__global__ __launch_bounds__(64 * kNormBwdWaves) void norm_bwd_kernel(NormParams p) {
  constexpr int CV = Vec<Elem>::kN;
  extern __shared__ float buf[];
  const Place a = place_of<Elem, kSteps>(p);
  const int64_t round = int64_t(blockDim.x >> 6) * (int64_t(CV) << p.lanes_log2);
  const int64_t base = int64_t(a.grp) * p.g;
  Square<Elem, kSteps> y, z, g;
  float w[CV], sum[kSteps], r[kSteps];
#pragma unroll
  for (int t = 0; t < kSteps; ++t) {
    sum[t] = 0.0f;
    r[t] = t < a.nt ? p.rstd[a.b * p.rb + a.grp * p.rg + (a.t0 + t) * p.rt] : 0.0f;
  }
  auto read = [&](int64_t c0) {
    const int nc = channels_left<CV>(p, c0);
    load_square<Elem, kSteps>(p.y, a.b, base + c0, a.t0, nc, a.nt, y);
    if constexpr (kMode != kNoGate) load_square<Elem, kSteps>(p.z, a.b, base + c0, a.t0, nc, a.nt, z);
    load_square<Elem, kSteps>(p.dout, a.b, base + c0, a.t0, nc, a.nt, g);
    load_run<float, CV>(p.weight + base + c0, nc, w);
  };
  // sum_G A v: w dout y s either way
  auto add = [&]() {
#pragma unroll
    for (int c = 0; c < CV; ++c)
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        float v = y.at(c, t);
        if constexpr (kMode != kNoGate) v *= silu_f(z.at(c, t));
        sum[t] = __builtin_fmaf(w[c] * g.at(c, t), v, sum[t]);
        if (kSteps > 1 && t == kSteps - 1) __builtin_amdgcn_sched_barrier(0);
      }
  };
  if constexpr (kHeld) {
    read(a.c0);
    add();
  } else {
    for (int k = 0; k < p.blocks; ++k) {
      read(a.c0 + k * round);
      add();
    }
  }
  sum_group<kSteps>(sum, p.lanes_log2, buf);
  float m[kSteps];  // r^3 S / G
#pragma unroll
  for (int t = 0; t < kSteps; ++t) m[t] = r[t] * r[t] * r[t] * (sum[t] * p.inv_g);

  auto write = [&](int64_t c0) {
    const int nc = channels_left<CV>(p, c0);
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
          const float zv = z.at(c, t), sg = sigmoid_f(zv);
          s = zv * sg;
          ds = sg * __builtin_fmaf(zv, 1.0f - sg, 1.0f);
        }
        dw[c] = __builtin_fmaf(gv * s, yv * r[t], dw[c]);
        const float a1 = r[t] * (w[c] * gv);
        if constexpr (kMode == kNormFirst) {
          dy[t] = __builtin_fmaf(-yv, m[t], a1 * s);
          dz[t] = a1 * yv * ds;
        } else {
          const float dv = __builtin_fmaf(-(yv * s), m[t], a1);
          dy[t] = dv * s;
          dz[t] = dv * yv * ds;
        }
      }
      put<Elem, kSteps>(dys, c, dy, row_y);
      if constexpr (kMode != kNoGate) put<Elem, kSteps>(dzs, c, dz, row_z);
      // A channel's words go out of use as its gradients' words come into it, if the channels
      // are not interleaved (nor its sums put off).
      if constexpr (kSteps > 1) {
        asm volatile("" : "+v"(dw[c]));
        forget_word(dys.w[c]);
        if constexpr (kMode != kNoGate) forget_word(dzs.w[c]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    store_square<Elem, kSteps>(p.dy, a.b, base + c0, a.t0, nc, a.nt, dys);
    if constexpr (kMode != kNoGate) store_square<Elem, kSteps>(p.dz, a.b, base + c0, a.t0, nc, a.nt, dzs);
    // over the lanes along time, then one store per channel
    for (int k = 32; k >= (1 << p.lanes_log2); k >>= 1)
#pragma unroll
      for (int c = 0; c < CV; ++c) dw[c] += __shfl_xor(dw[c], k, 64);
    if ((threadIdx.x & 63) < (1u << p.lanes_log2))
      store_run<float, CV>(p.part + (int64_t(a.b) * p.tiles + a.tile) * (int64_t(p.groups) * p.g) + base + c0,
                           nc, dw);
  };
  if constexpr (kHeld) {
    if constexpr (kSteps > 1) {
      forget<Elem, kSteps>(y);
      forget<Elem, kSteps>(g);
      if constexpr (kMode != kNoGate) forget<Elem, kSteps>(z);
    }
    write(a.c0);
  } else {
    for (int k = 0; k < p.blocks; ++k) {
      read(a.c0 + k * round);
      write(a.c0 + k * round);
    }
  }
}

constexpr int kReduceCols = 32, kReduceSlices = 32;

__global__ __launch_bounds__(kReduceCols* kReduceSlices) void norm_bwd_reduce(const float* part, float* dweight,
                                                                              int64_t rows, int64_t cols) {
  __shared__ float buf[kReduceSlices][kReduceCols + 1];
  const int64_t col = int64_t(blockIdx.x) * kReduceCols + threadIdx.x % kReduceCols;
  const float a = sum_rows<kReduceCols, kReduceSlices>(part, rows, cols, col, buf);
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
  p.blocks = int(s.blocks);
  p.norm_first = a.norm_first ? 1 : 0;
  p.tiles = uint32_t(s.tiles);
  p.total = uint32_t(s.tiles * a.groups * a.batch);
  return p;
}

template <typename Elem, int kSteps, bool kHeld, int kMode>
void launch(const NormParams& p, const NormShape& s, bool backward, hipStream_t st) {
  const dim3 grid(p.total), block(64 * s.waves);
  const size_t lds = size_t(s.waves) * (64 >> s.lanes_log2) * kSteps * 4;
  if constexpr (kSteps > 1) {  // (the backward has no form of one step)
    if (backward) {
      hipLaunchKernelGGL((norm_bwd_kernel<Elem, kSteps, kHeld, kMode>), grid, block, lds, st, p);
      return;
    }
  }
  hipLaunchKernelGGL((norm_fwd_kernel<Elem, kSteps, kHeld, kMode>), grid, block, lds, st, p);
}

template <typename Elem, int kSteps, bool kHeld>
void run_mode(const NormParams& p, const NormShape& s, bool backward, hipStream_t st) {
  if (!p.z.p)
    launch<Elem, kSteps, kHeld, kNoGate>(p, s, backward, st);
  else if (p.norm_first)
    launch<Elem, kSteps, kHeld, kNormFirst>(p, s, backward, st);
  else
    launch<Elem, kSteps, kHeld, kGateFirst>(p, s, backward, st);
}

template <typename Elem>
void run(const NormParams& p, const NormShape& s, bool backward, hipStream_t st) {
  constexpr int CV = Vec<Elem>::kN;
  if (s.steps == 1)
    s.blocks == 1 ? run_mode<Elem, 1, true>(p, s, backward, st) : run_mode<Elem, 1, false>(p, s, backward, st);
  else
    s.blocks == 1 ? run_mode<Elem, CV, true>(p, s, backward, st) : run_mode<Elem, CV, false>(p, s, backward, st);
}

}  // namespace

int launch_norm_fwd(const NormArgs& a, void* stream) {
  const bool chan = a.y.order == Order::Channel && (!a.z.p || a.z.order == Order::Channel) &&
                    a.out.order == Order::Channel;
  const NormShape s = norm_shape(a.dim, a.groups, a.seqlen, a.io, chan, kNormFwdWaves);
  const NormParams p = params_of(a, s);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (a.io == Io::BF16)
    run<uint16_t>(p, s, false, st);
  else
    run<float>(p, s, false, st);
  return int(hipGetLastError());
}

int launch_norm_bwd(const NormArgs& a, void* stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  int64_t rows = 0;
  if (a.batch > 0 && a.seqlen > 0) {
    const NormShape s = norm_bwd_shape(a.dim, a.groups, a.seqlen, a.io);
    const NormParams p = params_of(a, s);
    if (a.io == Io::BF16)
      run<uint16_t>(p, s, true, st);
    else
      run<float>(p, s, true, st);
    const int err = int(hipGetLastError());
    if (err) return err;
    rows = norm_partials(a.batch, s);
  }
  hipLaunchKernelGGL(norm_bwd_reduce, dim3(unsigned((a.dim + kReduceCols - 1) / kReduceCols)),
                     dim3(kReduceCols * kReduceSlices), 0, st, a.workspace, a.dweight, rows, a.dim);
  return int(hipGetLastError());
}

}  // namespace ssm
