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
// last lanes hold less. A row's lanes take several heads of the step in turn, all loads first, with
// the angles and weights loaded once.
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
  int heads;
};

struct QkParams {
  QkSide side[2];
  const float *cos, *sin;
  const int32_t* positions;
  float eps, inv_dim;
  float* partials;           // backward, nullable: [workgroups, 2, dim]
  int64_t items, seqlen, table_rows;
  int q_parts, parts, dim, rot, turning;  // turning: lanes of a row that hold pairs
  int interleaved;
};

// The two runs of a lane: values [a, a + na) and [b, b + nb), and its first angle.
struct Runs {
  int a, b, na, nb, angle;
  bool turns;
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

template <typename Elem>
__device__ __forceinline__ void store_runs(Elem* p, const Runs& u, const float (&v)[8]) {
  const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
  store_few<Elem, 4>(p + u.a, u.na, a);
  store_few<Elem, 4>(p + u.b, u.nb, b);
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

// One item: its side, heads, step and angles.
struct Item {
  int side, head0;
  int64_t b, t;
  bool live, at_table;
};

__device__ __forceinline__ Item item_of(int64_t at, const QkParams& p, int rows) {
  Item x;
  x.live = at < p.items;
  const int64_t step = (x.live ? at : 0) / p.parts;
  const int part = int((x.live ? at : 0) % p.parts);
  x.side = part >= p.q_parts ? 1 : 0;
  x.head0 = (x.side ? part - p.q_parts : part) * rows;
  x.b = step / p.seqlen;
  x.t = step % p.seqlen;
  return x;
}

__device__ __forceinline__ void load_angles(const QkParams& p, Item& x, const Runs& u, float (&c)[4], float (&s)[4]) {
  const int64_t pos = p.positions ? p.positions[x.b * p.seqlen + x.t] : x.t;
  x.at_table = p.rot == 0 || (pos >= 0 && pos < p.table_rows);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
  }
  if (u.turns && x.at_table) {
    const int half = p.rot / 2, n = half - u.angle;
    load_few<float, 4>(p.cos + pos * half + u.angle, n, c);
    load_few<float, 4>(p.sin + pos * half + u.angle, n, s);
  }
}

template <typename Elem, int LG, int R>
__global__ __launch_bounds__(kThreads) void qk_fwd_kernel(QkParams p) {
  const int lane = threadIdx.x & ((1 << LG) - 1);
  const int64_t at = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> LG;
  Item x = item_of(at, p, R);
  if (!x.live) return;
  const QkSide& d = p.side[x.side];
  const Runs u = runs_of(lane, p);
  const Elem* from = static_cast<const Elem*>(d.x) + x.b * d.batch + x.t * d.step + x.head0 * d.head;
  const int rows = d.heads - x.head0 < R ? d.heads - x.head0 : R;
  float v[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) load_runs<Elem>(from + (i < rows ? i : 0) * d.head, u, v[i]);
  float c[4], s[4], w[8];
  load_angles(p, x, u, c, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.0f;
  if (d.weight) load_runs<float>(d.weight, u, w);
  Elem* to = static_cast<Elem*>(d.out) + ((x.b * p.seqlen + x.t) * d.heads + x.head0) * p.dim;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(v[i][e], v[i][e], sum);
    const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum_lanes<LG>(sum), p.inv_dim, p.eps));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = v[i][e] * r * w[e];
    turn(v[i], c, s, p.interleaved != 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] = x.at_table ? v[i][e] : 0.0f;
    if (i < rows) store_runs<Elem>(to + i * p.dim, u, v[i]);
  }
}

template <typename Elem, int LG, int R>
__global__ __launch_bounds__(kThreads) void qk_bwd_kernel(QkParams p) {
  constexpr int kPer = kThreads >> LG;  // items of a workgroup at a time
  const int lane = threadIdx.x & ((1 << LG) - 1), mine = threadIdx.x >> LG;
  const Runs u = runs_of(lane, p);
  float w[2][8], dw[2][8];
#pragma unroll
  for (int side = 0; side < 2; ++side) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[side][e] = 1.0f;
      dw[side][e] = 0.0f;
    }
    if (p.side[side].weight) load_runs<float>(p.side[side].weight, u, w[side]);
  }
  for (int64_t first = int64_t(blockIdx.x) * kPer; first < p.items; first += int64_t(gridDim.x) * kPer) {
    Item x = item_of(first + mine, p, R);  // (past the last: the first item's values, not stored)
    const QkSide& d = p.side[x.side];
    const Elem* from = static_cast<const Elem*>(d.x) + x.b * d.batch + x.t * d.step + x.head0 * d.head;
    const Elem* dy = static_cast<const Elem*>(d.dy) + x.b * d.dy_batch + x.t * d.dy_step + x.head0 * d.dy_head;
    const int rows = !x.live ? 0 : d.heads - x.head0 < R ? d.heads - x.head0 : R;
    float v[R][8], y[R][8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      load_runs<Elem>(from + (i < rows ? i : 0) * d.head, u, v[i]);
      load_runs<Elem>(dy + (i < rows ? i : 0) * d.dy_head, u, y[i]);
    }
    float c[4], s[4];
    load_angles(p, x, u, c, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = -s[e];
    Elem* to = static_cast<Elem*>(d.out) + ((x.b * p.seqlen + x.t) * d.heads + x.head0) * p.dim;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      turn(y[i], c, s, p.interleaved != 0);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(v[i][e], v[i][e], sum);
      const float r = 1.0f / __builtin_sqrtf(__builtin_fmaf(sum_lanes<LG>(sum), p.inv_dim, p.eps));
      float dot = 0.0f;
      const bool counts = i < rows && x.at_table;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] *= r;
        const float add = y[i][e] * v[i][e], we = x.side ? w[1][e] : w[0][e];
        dw[0][e] += counts && !x.side ? add : 0.0f;
        dw[1][e] += counts && x.side ? add : 0.0f;
        dot = __builtin_fmaf(add, we, dot);
        y[i][e] *= we;
      }
      const float mean = sum_lanes<LG>(dot) * p.inv_dim;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = r * (y[i][e] - v[i][e] * mean);
        v[i][e] = x.at_table ? o : 0.0f;
      }
      if (i < rows) store_runs<Elem>(to + i * p.dim, u, v[i]);
    }
  }
  if (!p.partials) return;
  // The weight gradients of the workgroup's items, in the order of its lane groups.
  __shared__ float part[kPer][8 << LG];
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) part[mine][lane * 8 + e] = side ? dw[1][e] : dw[0][e];
    __syncthreads();
    if (threadIdx.x < (1 << LG)) {
      float a[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = 0.0f;
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += part[i][lane * 8 + e];
      float* to = p.partials + (int64_t(blockIdx.x) * 2 + side) * p.dim;
      store_runs<float>(to, u, a);
    }
  }
}

// The workgroups' partial weight gradients summed, in a fixed order.
__global__ __launch_bounds__(kReduceCols* kNormReduceSlices) void qk_weight_kernel(const float* part, int64_t rows,
                                                                                   int dim, float* dq_weight,
                                                                                   float* dk_weight) {
  __shared__ float buf[kNormReduceSlices][kReduceCols + 1];
  const int64_t col = int64_t(blockIdx.x) * kReduceCols + threadIdx.x % kReduceCols, cols = 2 * dim;
  const float a = sum_rows<kReduceCols, kNormReduceSlices>(part, rows, cols, col, buf);
  if (threadIdx.x / kReduceCols == 0 && col < cols) {
    float* to = col < dim ? dq_weight : dk_weight;
    if (to) to[col < dim ? col : col - dim] = a;
  }
}

template <typename Elem, int LG, int R>
void run(const QkParams& p, bool bwd, int64_t groups, hipStream_t s) {
  const dim3 grid{uint32_t(groups)}, block{kThreads};
  if (bwd)
    hipLaunchKernelGGL((qk_bwd_kernel<Elem, LG, R>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((qk_fwd_kernel<Elem, LG, R>), grid, block, 0, s, p);
}

template <typename Elem, int R>
void run_lanes(const QkParams& p, int lg, bool bwd, int64_t groups, hipStream_t s) {
  switch (lg) {
    case 2: return run<Elem, 2, R>(p, bwd, groups, s);
    case 3: return run<Elem, 3, R>(p, bwd, groups, s);
    case 4: return run<Elem, 4, R>(p, bwd, groups, s);
    case 5: return run<Elem, 5, R>(p, bwd, groups, s);
    default: return run<Elem, 6, R>(p, bwd, groups, s);
  }
}

int launch(const QkArgs& a, bool bwd, void* stream) {
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int lg = qk_lanes_log2(a.dim, a.rot), rows = qk_rows(a.batch, a.seqlen, a.q_heads + a.k_heads, lg);
  const QkItems items = qk_items(a.batch, a.seqlen, a.q_heads, a.k_heads, rows);
  const int64_t all = qk_groups(items.items, lg), groups = bwd ? qk_partials(all) : all;
  const bool sums = bwd && (a.dq_weight || a.dk_weight);
  QkParams p{};
  p.side[0] = QkSide{a.q.p, a.q.batch, a.q.step, a.q.head, a.dyq.p, a.dyq.batch, a.dyq.step, a.dyq.head,
                     a.q_weight, a.q_out, int(a.q_heads)};
  p.side[1] = QkSide{a.k.p, a.k.batch, a.k.step, a.k.head, a.dyk.p, a.dyk.batch, a.dyk.step, a.dyk.head,
                     a.k_weight, a.k_out, int(a.k_heads)};
  p.cos = a.cos, p.sin = a.sin, p.positions = a.positions;
  p.eps = a.eps, p.inv_dim = 1.0f / float(a.dim);
  p.partials = sums ? a.workspace : nullptr;
  p.items = items.items, p.seqlen = a.seqlen, p.table_rows = a.table_rows;
  p.q_parts = int(items.q_parts), p.parts = int(items.q_parts + items.k_parts);
  p.dim = int(a.dim), p.rot = int(a.rot), p.turning = int((a.rot / 2 + 3) / 4);
  p.interleaved = a.interleaved;
  if (groups > 0) {
    if (a.io == Io::BF16) {
      if (rows > 1) run_lanes<uint16_t, kQkMostRows>(p, lg, bwd, groups, s);
      else run_lanes<uint16_t, 1>(p, lg, bwd, groups, s);
    } else {
      if (rows > 1) run_lanes<float, kQkMostRows>(p, lg, bwd, groups, s);
      else run_lanes<float, 1>(p, lg, bwd, groups, s);
    }
    if (hipGetLastError() != hipSuccess) return -1;
  }
  if (sums) {
    hipLaunchKernelGGL(qk_weight_kernel, dim3(uint32_t(reduce_groups(2 * a.dim))),
                       dim3(kReduceCols * kNormReduceSlices), 0, s, a.workspace, groups, int(a.dim), a.dq_weight,
                       a.dk_weight);
    if (hipGetLastError() != hipSuccess) return -1;
  }
  return 0;
}

}  // namespace

int launch_qk_fwd(const QkArgs& a, void* stream) { return launch(a, false, stream); }
int launch_qk_bwd(const QkArgs& a, void* stream) { return launch(a, true, stream); }

}  // namespace ssm
