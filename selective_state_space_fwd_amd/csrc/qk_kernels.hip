// RMS norm of every head's queries and keys with the position rotation in the same pass, and its
// gradient, on gfx950 (include/ssm_qk.h).
//
//   n = x r, r = 1 / sqrt(mean(x^2) + eps);  y = w n;  out = y with pairs (a, b) of its first rot values
//   turned: (a cos - b sin, b cos + a sin)
//   dy = dout turned back;  dx = r (w dy - n mean(w dy n));  dw = sum dy n
//
// Memory binds it: each value is read once and written once (the gradient: read twice, written
// once). A row is one head of one step; its lanes hold eight values each as two runs of four, which
// are four whole pairs in either pairing: the runs at i and i + rot / 2 (halves), or eight
// neighbours. So a rotation needs no other lane, and whatever rot and dim are, only the
// last lanes hold less. In large calls a row's lanes take several heads of the step together, all loads
// first, with the angles and weights loaded once; the gradient's workgroups stay for many items, the
// next one's loads on their way, and leave one row of weight gradients each.
//
// Measured, b4 2048 steps of 32 + 8 heads of 128 in bf16, inputs not in cache: forward 33.4 us for 168.8 MB
// (5.1 TB/s, a copy's rate; the values are held as they came until all heads' loads are out, 38 us widened at
// once), gradient with its weights' sum 65.4 us for 252.7 MB (3.9 TB/s). b8 one token: 5 to 6 us, what a launch
// costs.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_block.h"
#include "qk_launch.h"

namespace ssm {
namespace {

constexpr int kThreads = 64 * kQkWaves;

struct QkSide {
  const void* x;
  int64_t batch, step, head;
  const void* dy;
  int64_t dy_batch, dy_step, dy_head;
  const float* weight;
  void* out;
  float* partials;           // backward, nullable: [workgroups, dim]
  uint32_t items, parts;     // all, and of a step
  int heads;
};

struct QkParams {
  QkSide side[2];
  uint32_t q_groups;         // workgroups of q, before those of k
  const float *cos, *sin;
  const int32_t* positions;
  float eps, inv_dim;
  uint32_t places;           // positions from here on, and those below 0, are padding
  uint32_t seqlen;
  int dim, rot, turning;     // turning: lanes of a row that hold pairs
  int interleaved;
};

// The two runs of a lane: values [a, a + na) and [b, b + nb), and its first angle.
struct Runs {
  int a, b, na, nb, angle;
  bool turns, joined;      // joined: eight neighbours, all there
};

__device__ __forceinline__ int clamp4(int n) { return n < 0 ? 0 : n > 4 ? 4 : n; }

__device__ __forceinline__ Runs runs_of(int unit, const QkParams& p) {
  Runs u;
  u.turns = unit < p.turning;
  u.angle = 4 * unit;
  if (u.turns && !p.interleaved) {
    u.a = 4 * unit;
    u.b = p.rot / 2 + 4 * unit;
    u.na = u.nb = clamp4(p.rot / 2 - 4 * unit);
  } else {
    u.a = u.turns ? 8 * unit : p.rot + 8 * (unit - p.turning);
    u.b = u.a + 4;
    const int n = (u.turns ? p.rot : p.dim) - u.a;
    u.na = clamp4(n);
    u.nb = clamp4(n - 4);
  }
  u.joined = u.b == u.a + 4 && u.nb == 4;
  return u;
}

template <typename Elem>
__device__ __forceinline__ void load_runs(const Elem* p, const Runs& u, float (&v)[8]) {
  float a[4], b[4];
  load_few<Elem, 4>(p + u.a, u.na, a);
  load_few<Elem, 4>(p + u.b, u.nb, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

// The runs as they stand in memory, to be widened when their turn comes.
template <typename Elem>
struct RawRuns {
  Dwords<int(sizeof(Elem))> a, b;
};

template <typename Elem>
__device__ __forceinline__ Dwords<int(sizeof(Elem))> load_raw4(const Elem* p, int n) {
  using Raw = Dwords<int(sizeof(Elem))>;
  if (n >= 4) return *reinterpret_cast<const Raw*>(p);
  float v[4];
  load_few<Elem, 4>(p, n, v);
  Raw d;
  pack_few<Elem, 4>(v, d);
  return d;
}

template <typename Elem>
__device__ __forceinline__ RawRuns<Elem> load_raw(const Elem* p, const Runs& u) {
  if (sizeof(Elem) == 2 && u.joined) return *reinterpret_cast<const RawRuns<Elem>*>(p + u.a);
  return RawRuns<Elem>{load_raw4<Elem>(p + u.a, u.na), load_raw4<Elem>(p + u.b, u.nb)};
}

template <typename Elem>
__device__ __forceinline__ void widen_runs(const RawRuns<Elem>& d, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = few_elem<Elem>(d.a, i);
    v[4 + i] = few_elem<Elem>(d.b, i);
  }
}

// C values (n of them), past L2 with `stream`.
template <typename Elem, int C>
__device__ __forceinline__ void store_run_of(Elem* p, int n, const float (&v)[C], bool stream) {
  if (stream && n >= C) {
    Dwords<C * int(sizeof(Elem)) / 4> d;
    pack_few<Elem, C>(v, d);
    store_stream(p, d);
  } else {
    store_few<Elem, C>(p, n, v);
  }
}

template <typename Elem>
__device__ __forceinline__ void store_runs(Elem* p, const Runs& u, const float (&v)[8], bool stream) {
  if constexpr (sizeof(Elem) == 2) {
    if (u.joined) return store_run_of<Elem, 8>(p + u.a, 8, v, stream);
  }
  const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
  store_run_of<Elem, 4>(p + u.a, u.na, a, stream);
  store_run_of<Elem, 4>(p + u.b, u.nb, b, stream);
}

// Whether a store of the row's lanes fills lines; parts of lines go through L2, which joins them (8192 steps of
// 32 + 8 heads, past L2 | through it: fp32 heads of 128, neighbouring pairs 96.9 | 65.1 us; bf16 heads of 16 22.2 |
// 10.6; whole lines, bf16 heads of 128: 33.4 | 44).
template <typename Elem>
__device__ __forceinline__ bool fills_lines(const Runs& u, const QkParams& p) {
  return u.joined ? sizeof(Elem) == 2 : p.rot / 2 * int(sizeof(Elem)) >= 128;
}

// The four pairs turned by (c, s); by (c, -s) for the way back.
__device__ __forceinline__ void turn(float (&v)[8], const float (&c)[4], const float (&s)[4], bool interleaved) {
  float o[8];
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = v[2 * i] * c[i] - v[2 * i + 1] * s[i];
      o[2 * i + 1] = v[2 * i + 1] * c[i] + v[2 * i] * s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = v[i] * c[i] - v[4 + i] * s[i];
      o[4 + i] = v[4 + i] * c[i] + v[i] * s[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = o[i];
}

// One item: its heads, step and angles.
struct Item {
  uint32_t b, t;
  int head0;
  bool live, at_table;
};

__device__ __forceinline__ Item item_of(uint32_t at, const QkSide& d, uint32_t seqlen, int rows) {
  Item x;
  x.live = at < d.items;
  at = x.live ? at : 0;
  const uint32_t step = at / d.parts;
  x.head0 = int(at - step * d.parts) * rows;
  x.b = step / seqlen;
  x.t = step - x.b * seqlen;
  return x;
}

__device__ __forceinline__ void load_angles(const QkParams& p, Item& x, const Runs& u, float (&c)[4], float (&s)[4]) {
  const uint32_t pos = p.positions ? uint32_t(p.positions[int64_t(x.b) * p.seqlen + x.t]) : x.t;
  x.at_table = pos < p.places;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  if (u.turns && x.at_table) {
    const int half = p.rot / 2, n = half - u.angle;
    load_few<float, 4>(p.cos + int64_t(pos) * half + u.angle, n, c);
    load_few<float, 4>(p.sin + int64_t(pos) * half + u.angle, n, s);
  }
}

template <typename Elem, int LG, bool kMany>
__global__ __launch_bounds__(kThreads) void qk_fwd_kernel(QkParams p) {
  constexpr int R = kMany ? qk_most_rows(false, sizeof(Elem)) : 1;
  constexpr uint32_t kPer = kThreads >> LG;  // items of a workgroup
  const int lane = threadIdx.x & ((1 << LG) - 1);
  const int side = blockIdx.x >= p.q_groups ? 1 : 0;
  const QkSide& d = p.side[side];
  const uint32_t group = blockIdx.x - (side ? p.q_groups : 0);
  Item x = item_of(group * kPer + (threadIdx.x >> LG), d, p.seqlen, R);
  if (!x.live) return;
  const Runs u = runs_of(lane, p);
  const bool stream = kMany && fills_lines<Elem>(u, p);
  const Elem* from = static_cast<const Elem*>(d.x) + x.b * d.batch + x.t * d.step + x.head0 * d.head;
  const int rows = d.heads - x.head0 < R ? d.heads - x.head0 : R;
  RawRuns<Elem> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i] = load_raw<Elem>(from + (i < rows ? i : 0) * d.head, u);
  float c[4], s[4], w[8];
  load_angles(p, x, u, c, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.0f;
  if (d.weight) load_runs<float>(d.weight, u, w);
  Elem* to = static_cast<Elem*>(d.out) + ((int64_t(x.b) * p.seqlen + x.t) * d.heads + x.head0) * p.dim;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float v[8];
    widen_runs<Elem>(raw[i], v);
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(v[e], v[e], sum);
    const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum_lanes<LG>(sum), p.inv_dim, p.eps));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[e];
    turn(v, c, s, p.interleaved != 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x.at_table ? v[e] : 0.0f;
    if (i < rows) store_runs<Elem>(to + i * p.dim, u, v, stream);
  }
}

template <typename Elem, int LG, bool kMany>
__global__ __launch_bounds__(kThreads, 4) void qk_bwd_kernel(QkParams p, uint32_t groups) {
  constexpr int R = kMany ? qk_most_rows(true, sizeof(Elem)) : 1;
  constexpr uint32_t kPer = kThreads >> LG;  // items of a workgroup at a time
  const int lane = threadIdx.x & ((1 << LG) - 1), mine = threadIdx.x >> LG;
  const int side = blockIdx.x >= p.q_groups ? 1 : 0;
  const QkSide& d = p.side[side];
  const uint32_t group = blockIdx.x - (side ? p.q_groups : 0), step = (side ? groups - p.q_groups : p.q_groups) * kPer;
  const Runs u = runs_of(lane, p);
  const bool stream = kMany && fills_lines<Elem>(u, p);
  float w[8], dw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[e] = 1.0f;
    dw[e] = 0.0f;
  }
  if (d.weight) load_runs<float>(d.weight, u, w);
  // What the next item reads is on its way while this one is worked on.
  Item next;
  RawRuns<Elem> next_v[R], next_y[R];
  float next_c[4], next_s[4];
  const auto load = [&](uint32_t first) {
    next = item_of(first + mine, d, p.seqlen, R);  // (past the last: the first item's values, not stored)
    const Elem* from = static_cast<const Elem*>(d.x) + next.b * d.batch + next.t * d.step + next.head0 * d.head;
    const Elem* dy = static_cast<const Elem*>(d.dy) + next.b * d.dy_batch + next.t * d.dy_step + next.head0 * d.dy_head;
    load_angles(p, next, u, next_c, next_s);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int row = next.head0 + i < d.heads ? i : 0;
      const Elem *xr = from + row * d.head, *yr = dy + row * d.dy_head;
      next_v[i] = RawRuns<Elem>{load_raw4<Elem>(xr + u.a, u.na), load_raw4<Elem>(xr + u.b, u.nb)};
      next_y[i] = RawRuns<Elem>{load_raw4<Elem>(yr + u.a, u.na), load_raw4<Elem>(yr + u.b, u.nb)};
    }
  };
  load(group * kPer);
  for (uint32_t first = group * kPer; first < d.items; first += step) {
    const Item x = next;
    const int rows = !x.live ? 0 : d.heads - x.head0 < R ? d.heads - x.head0 : R;
    RawRuns<Elem> raw_v[R], raw_y[R];
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      raw_v[i] = next_v[i];
      raw_y[i] = next_y[i];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = next_c[e];
      s[e] = -next_s[e];
    }
    load(first + step < d.items ? first + step : d.items);
    Elem* to = static_cast<Elem*>(d.out) + ((int64_t(x.b) * p.seqlen + x.t) * d.heads + x.head0) * p.dim;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float v[8], y[8];
      widen_runs<Elem>(raw_v[i], v);
      widen_runs<Elem>(raw_y[i], y);
      turn(y, c, s, p.interleaved != 0);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(v[e], v[e], sum);
      const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum_lanes<LG>(sum), p.inv_dim, p.eps));
      float dot = 0.0f;
      const bool counts = i < rows && x.at_table;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] *= r;
        const float add = y[e] * v[e];
        dw[e] += counts ? add : 0.0f;
        dot = __builtin_fmaf(add, w[e], dot);
        y[e] *= w[e];
      }
      const float mean = sum_lanes<LG>(dot) * p.inv_dim;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = r * (y[e] - v[e] * mean);
        v[e] = x.at_table ? o : 0.0f;
      }
      if (i < rows) store_runs<Elem>(to + i * p.dim, u, v, stream);
    }
  }
  if (!d.partials) return;
  // The weight gradient of the workgroup's items, in the order of its lane groups.
  __shared__ float part[kPer][8 << LG];
#pragma unroll
  for (int e = 0; e < 8; ++e) part[mine][lane * 8 + e] = dw[e];
  __syncthreads();
  if (threadIdx.x < (1 << LG)) {
    float a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = 0.0f;
    // (a few at a time: all at once would be the kernel's most registers)
#pragma unroll 4
    for (uint32_t i = 0; i < kPer; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] += part[i][lane * 8 + e];
    store_runs<float>(d.partials + int64_t(group) * p.dim, u, a, false);
  }
}

// The workgroups' partial weight gradients of a side summed, in a fixed order; a side the grid's
// second axis.
struct WeightSum {
  const float* part;
  int64_t rows;
  float* to;  // nullable
};
__global__ __launch_bounds__(kReduceCols* kNormReduceSlices) void qk_weight_kernel(WeightSum q, WeightSum k, int dim) {
  __shared__ float buf[kNormReduceSlices][kReduceCols + 1];
  const WeightSum& w = blockIdx.y ? k : q;
  if (!w.to) return;
  const int64_t col = int64_t(blockIdx.x) * kReduceCols + threadIdx.x % kReduceCols;
  const float a = sum_rows<kReduceCols, kNormReduceSlices>(w.part, w.rows, dim, col, buf);
  if (threadIdx.x / kReduceCols == 0 && col < dim) w.to[col] = a;
}

template <typename Elem, int LG>
void run(const QkParams& p, bool many, bool bwd, uint32_t groups, hipStream_t s) {
  const dim3 grid{groups}, block{kThreads};
  if (bwd && many)
    hipLaunchKernelGGL((qk_bwd_kernel<Elem, LG, true>), grid, block, 0, s, p, groups);
  else if (bwd)
    hipLaunchKernelGGL((qk_bwd_kernel<Elem, LG, false>), grid, block, 0, s, p, groups);
  else if (many)
    hipLaunchKernelGGL((qk_fwd_kernel<Elem, LG, true>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((qk_fwd_kernel<Elem, LG, false>), grid, block, 0, s, p);
}

template <typename Elem>
void run_lanes(const QkParams& p, int lg, bool many, bool bwd, uint32_t groups, hipStream_t s) {
  switch (lg) {
    case 2: return run<Elem, 2>(p, many, bwd, groups, s);
    case 3: return run<Elem, 3>(p, many, bwd, groups, s);
    case 4: return run<Elem, 4>(p, many, bwd, groups, s);
    case 5: return run<Elem, 5>(p, many, bwd, groups, s);
    default: return run<Elem, 6>(p, many, bwd, groups, s);
  }
}

int launch(const QkArgs& a, bool bwd, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int lg = qk_lanes_log2(a.dim, a.rot);
  const bool many = qk_many(a.batch, a.seqlen, a.q_heads + a.k_heads, lg);
  const int rows = many ? qk_most_rows(bwd, a.io == Io::BF16 ? 2 : 4) : 1;
  const int64_t q_items = qk_items(a.batch, a.seqlen, a.q_heads, rows),
                k_items = qk_items(a.batch, a.seqlen, a.k_heads, rows);
  int64_t q_groups = qk_groups(q_items, lg), k_groups = qk_groups(k_items, lg);
  if (bwd) {
    const int64_t q_all = q_groups;
    q_groups = qk_partials(q_all, k_groups);
    k_groups = qk_partials(k_groups, q_all);
  }
  const int64_t groups = q_groups + k_groups;
  float *q_part = a.workspace, *k_part = a.workspace ? a.workspace + q_groups * a.dim : nullptr;
  QkParams p{};
  p.side[0] = QkSide{a.q.p, a.q.batch, a.q.step, a.q.head, a.dyq.p, a.dyq.batch, a.dyq.step, a.dyq.head, a.q_weight,
                     a.q_out, a.dq_weight ? q_part : nullptr, uint32_t(q_items),
                     uint32_t((a.q_heads + rows - 1) / rows), int(a.q_heads)};
  p.side[1] = QkSide{a.k.p, a.k.batch, a.k.step, a.k.head, a.dyk.p, a.dyk.batch, a.dyk.step, a.dyk.head, a.k_weight,
                     a.k_out, a.dk_weight ? k_part : nullptr, uint32_t(k_items),
                     uint32_t((a.k_heads + rows - 1) / rows), int(a.k_heads)};
  p.q_groups = uint32_t(q_groups);
  p.cos = a.cos, p.sin = a.sin, p.positions = a.positions;
  p.eps = a.eps, p.inv_dim = 1.0f / float(a.dim);
  p.seqlen = uint32_t(a.seqlen);
  // (without a rotation there is no table, and every position that is not below 0 has a place)
  constexpr int64_t kMost = int64_t(1) << 31;
  p.places = uint32_t(a.rot == 0 || a.table_rows > kMost ? kMost : a.table_rows);
  p.dim = int(a.dim), p.rot = int(a.rot), p.turning = int((a.rot / 2 + 3) / 4);
  p.interleaved = a.interleaved;
  if (groups > 0) {
    const uint32_t n = uint32_t(groups);
    if (a.io == Io::BF16) run_lanes<uint16_t>(p, lg, many, bwd, n, s);
    else run_lanes<float>(p, lg, many, bwd, n, s);
    if (hipGetLastError() != hipSuccess) return -1;
  }
  if (bwd && (a.dq_weight || a.dk_weight)) {
    hipLaunchKernelGGL(qk_weight_kernel, dim3(uint32_t(reduce_groups(a.dim)), 2),
                       dim3(kReduceCols * kNormReduceSlices), 0, s, WeightSum{q_part, q_groups, a.dq_weight},
                       WeightSum{k_part, k_groups, a.dk_weight}, int(a.dim));
    if (hipGetLastError() != hipSuccess) return -1;
  }
  return 0;
}

}  // namespace

int launch_qk_fwd(const QkArgs& a, void* stream) { return launch(a, false, stream); }
int launch_qk_bwd(const QkArgs& a, void* stream) { return launch(a, true, stream); }

}  // namespace ssm
