// One step of the selective recurrence against a cache of states on gfx950
// (include/ssm_step.h): Mamba-1 (A per channel and state) and Mamba-2 (A and step size per
// head), for a batch of rows that each name a slot of the cache.
//
//   dt = softplus(dt + bias);  h = exp(dt A) h + dt x B;  y = sum_n C h + D x;  out = y silu(z)
//
// The state, fp32, is all of the traffic (8 bytes a state against 2 or 4 per channel), so the
// layout is the state's: a lane holds four consecutive states (16 bytes) of kCh channels, a
// channel's lanes are consecutive and a power of two in number, and every load of a wave is
// issued before the first use. y is the sum over a channel's lanes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_launch.h"
#include "device_block.h"

namespace ssm {
namespace {

constexpr int kWaves = 4;
constexpr int kCh = 4;  // channels per lane

struct StepParams {
  const void* x;
  const void* dt;
  const void* B;
  const void* C;
  const void* z;
  int64_t xs, dts, bs, cs, zs;
  const float* A;
  const float* D;
  const float* bias;
  float* state;
  const int32_t* slots;
  void* out;
  int64_t nslots;
  int batch, dim, dstate, headdim, softplus;
};

// Four states from p on, those at and past n zero (not read).
__device__ __forceinline__ void load4(const float* p, int n, float (&v)[4]) {
  load_run<float, 4>(p, n, v);
}

template <typename Elem>
__device__ __forceinline__ void load4_row(const void* base, int64_t off, int n, float (&v)[4]) {
  const Elem* p = static_cast<const Elem*>(base) + off;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < n ? widen<Elem>(p[i]) : 0.0f;
}

// LG: log2 of the lanes per channel.
template <typename Elem, int LG, bool kHeads>
__global__ __launch_bounds__(64 * kWaves) void state_step_kernel(StepParams p) {
  constexpr int CPW = 64 >> LG;  // channels per wave and access
  const int lane = threadIdx.x & 63;
  const int wave = blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int n0 = (lane & ((1 << LG) - 1)) * 4;
  const int nn = p.dstate - n0 < 4 ? p.dstate - n0 : 4;  // states of this lane (<= 0: none)
  const int64_t first_ch = int64_t(wave) * kCh * CPW + (lane >> LG);
  int r = blockIdx.y;
  const int slot = p.slots ? p.slots[r] : r;
  if (slot < 0 || slot >= p.nslots) {  // a row of no slot: zeros
#pragma unroll
    for (int k = 0; k < kCh; ++k) {
      const int64_t ch = first_ch + k * CPW;
      if (n0 == 0 && ch < p.dim) static_cast<Elem*>(p.out)[int64_t(r) * p.dim + ch] = Elem(0);
    }
    return;
  }
  float h[kCh][4], a[kCh][4];
#pragma unroll
  for (int k = 0; k < kCh; ++k) {
    const int64_t ch = first_ch + k * CPW;
    const int n = ch < p.dim ? nn : 0;
    load4(p.state + (int64_t(slot) * p.dim + ch) * p.dstate + n0, n, h[k]);
    if constexpr (kHeads) {
      a[k][0] = ch < p.dim ? p.A[uint32_t(ch) / uint32_t(p.headdim)] * kLog2e : 0.0f;
    } else {
      load4(p.A + ch * p.dstate + n0, n, a[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[k][i] *= kLog2e;
    }
  }
  SlotOrder order{true, INT32_MAX};
  if (p.slots) order = slot_order(p.slots, p.batch, r, slot);
  if (!order.first) return;
  for (;;) {
    float bv[4], cv[4], x[kCh], y[kCh];
    load4_row<Elem>(p.B, r * p.bs + n0, nn, bv);
    load4_row<Elem>(p.C, r * p.cs + n0, nn, cv);
#pragma unroll
    for (int k = 0; k < kCh; ++k) {
      const int64_t ch = first_ch + k * CPW;
      const bool ok = ch < p.dim;
      const int64_t step = kHeads ? int64_t(uint32_t(ok ? ch : 0) / uint32_t(p.headdim)) : ch;
      x[k] = ok ? widen<Elem>(static_cast<const Elem*>(p.x)[r * p.xs + ch]) : 0.0f;
      float dt = ok ? widen<Elem>(static_cast<const Elem*>(p.dt)[r * p.dts + step]) : 0.0f;
      if (ok && p.bias) dt += p.bias[step];
      if (p.softplus) dt = softplus_f(dt);
      const float dx = dt * x[k];
      const float one = kHeads ? exp2_hw(dt * a[k][0]) : 0.0f;
      y[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float keep = kHeads ? one : exp2_hw(dt * a[k][i]);
        h[k][i] = __builtin_fmaf(keep, h[k][i], dx * bv[i]);
        // (a lane's states past dstate add nothing, whatever dt x is)
        y[k] = i < nn ? __builtin_fmaf(cv[i], h[k][i], y[k]) : y[k];
      }
    }
#pragma unroll
    for (int k = 0; k < kCh; ++k) y[k] = sum_lanes<LG>(y[k]);
#pragma unroll
    for (int k = 0; k < kCh; ++k) {
      const int64_t ch = first_ch + k * CPW;
      if (n0 == 0 && ch < p.dim) {
        float v = p.D ? __builtin_fmaf(p.D[ch], x[k], y[k]) : y[k];
        if (p.z) v = gate_f(v, widen<Elem>(static_cast<const Elem*>(p.z)[r * p.zs + ch]));
        static_cast<Elem*>(p.out)[int64_t(r) * p.dim + ch] = narrow<Elem>(v);
      }
    }
    if (order.next == INT32_MAX) break;
    r = order.next;
    order = slot_order(p.slots, p.batch, r, slot);
  }
#pragma unroll
  for (int k = 0; k < kCh; ++k) {
    const int64_t ch = first_ch + k * CPW;
    const int n = ch < p.dim ? nn : 0;
    store_run<float, 4>(p.state + (int64_t(slot) * p.dim + ch) * p.dstate + n0, n, h[k]);
  }
}

template <typename Elem, int LG>
void run_lg(const StepArgs& a, const StepParams& p, hipStream_t s) {
  constexpr int per = kWaves * kCh * (64 >> LG);
  const dim3 grid(unsigned((a.dim + per - 1) / per), unsigned(a.batch));
  if (a.headdim)
    hipLaunchKernelGGL((state_step_kernel<Elem, LG, true>), grid, dim3(64 * kWaves), 0, s, p);
  else
    hipLaunchKernelGGL((state_step_kernel<Elem, LG, false>), grid, dim3(64 * kWaves), 0, s, p);
}

template <typename Elem>
void run(const StepArgs& a, const StepParams& p, hipStream_t s) {
  int lg = 0;
  while ((int64_t(4) << lg) < a.dstate) ++lg;  // dstate <= 256, so lg <= 6
  switch (lg) {
    case 0: return run_lg<Elem, 0>(a, p, s);
    case 1: return run_lg<Elem, 1>(a, p, s);
    case 2: return run_lg<Elem, 2>(a, p, s);
    case 3: return run_lg<Elem, 3>(a, p, s);
    case 4: return run_lg<Elem, 4>(a, p, s);
    case 5: return run_lg<Elem, 5>(a, p, s);
    default: return run_lg<Elem, 6>(a, p, s);
  }
}

}  // namespace

int launch_state_step(const StepArgs& a, void* stream) {
  StepParams p{a.x, a.dt, a.B, a.C, a.z, a.x_stride, a.dt_stride, a.b_stride, a.c_stride,
               a.z_stride, a.A, a.D, a.dt_bias, a.state, a.slots, a.out, a.nslots, int(a.batch),
               int(a.dim), int(a.dstate), int(a.headdim), a.softplus ? 1 : 0};
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.io == Io::BF16)
    run<uint16_t>(a, p, s);
  else
    run<float>(a, p, s);
  return int(hipGetLastError());
}

}  // namespace ssm
