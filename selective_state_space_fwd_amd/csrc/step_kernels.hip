// One step of the selective recurrence against a cache of states on gfx950
// (include/ssm_step.h): Mamba-1 (A per channel and state) and Mamba-2 (A and step size per
// head), for a batch of rows that each name a slot of the cache.
//
//   dt = softplus(dt + bias);  h = exp(dt A) h + dt x B;  y = sum_n C h + D x;  out = y silu(z)
//
// The state, fp32, is all of the traffic (8 bytes a state against 2 or 4 per channel), so the
// layout is the state's: a lane holds four consecutive states (16 bytes) of CH channels, a
// channel's lanes are consecutive and a power of two in number. What there is one of per
// channel (x, the step size, D, z) is loaded by one lane per channel of the wave, in one
// access each, and dealt to the channel's lanes through the LDS crossbar; y, the sum over a
// channel's lanes, goes back the same way, so that out is one access too. No load waits for
// another but the state's for its slot.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "block_launch.h"
#include "device_block.h"

namespace ssm {
namespace {

constexpr int kWaves = kStepWaves;

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

// Four states from p on, those at and past n zero (not read), and back. kStream: past the
// caches (non-temporal).
template <bool kStream>
__device__ __forceinline__ void load4(const float* p, int n, float (&v)[4]) {
  if constexpr (kStream) {
    typedef float quad __attribute__((ext_vector_type(4), aligned(4)));
    if (n >= 4) {
      const quad q = __builtin_nontemporal_load(reinterpret_cast<const quad*>(p));
      v[0] = q.x;
      v[1] = q.y;
      v[2] = q.z;
      v[3] = q.w;
      return;
    }
  }
  load_run<float, 4>(p, n, v);
}

template <bool kStream>
__device__ __forceinline__ void store4(float* p, int n, const float (&v)[4]) {
  if (kStream && n >= 4)
    store_run_stream<float, 4>(p, n, v);
  else
    store_run<float, 4>(p, n, v);
}

template <typename Elem>
__device__ __forceinline__ void load4_row(const void* base, int64_t off, int n, float (&v)[4]) {
  const Elem* p = static_cast<const Elem*>(base) + off;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = i < n ? widen<Elem>(p[i]) : 0.0f;
}

// What a lane holds for its one channel of the wave's (lanes past the wave's channels: zeros).
struct Channel {
  float x, dt, z;
};

// LG: log2 of the lanes per channel. CH: channels per lane, at most 2^LG (a lane per channel).
template <typename Elem, int LG, int CH, bool kHeads, bool kStream>
__global__ __launch_bounds__(64 * kWaves) void state_step_kernel(StepParams p) {
  constexpr int CPW = 64 >> LG;  // channels per wave and access
  static_assert(CH * CPW <= 64, "a lane per channel");
  const int lane = threadIdx.x & 63;
  const int wave = blockIdx.x * kWaves + (threadIdx.x >> 6);
  const int n0 = (lane & ((1 << LG) - 1)) * 4;
  const int nn = p.dstate - n0 < 4 ? p.dstate - n0 : 4;  // states of this lane (<= 0: none)
  const int64_t ch0 = int64_t(wave) * (CH * CPW);        // the wave's first channel
  const int64_t mine = ch0 + lane;                       // this lane's one channel
  const bool own = lane < CH * CPW && mine < p.dim;
  const int64_t first_ch = ch0 + (lane >> LG);           // of its states, the first
  int r = blockIdx.y;
  const int slot = p.slots ? p.slots[r] : r;

  const int64_t step = kHeads ? int64_t(uint32_t(own ? mine : 0) / uint32_t(p.headdim)) : mine;
  auto load_channel = [&](int row) {
    Channel c{0.0f, 0.0f, 0.0f};
    if (own) {
      c.x = widen<Elem>(static_cast<const Elem*>(p.x)[row * p.xs + mine]);
      c.dt = widen<Elem>(static_cast<const Elem*>(p.dt)[row * p.dts + step]);
      if (p.z) c.z = widen<Elem>(static_cast<const Elem*>(p.z)[row * p.zs + mine]);
    }
    return c;
  };
  Channel c = load_channel(r);
  const float bias = own && p.bias ? p.bias[step] : 0.0f;
  const float skip = own && p.D ? p.D[mine] : 0.0f;
  const float head_a = kHeads && own ? p.A[step] * kLog2e : 0.0f;
  float bv[4], cv[4], a[kHeads ? 1 : CH][4], h[CH][4];
  load4_row<Elem>(p.B, r * p.bs + n0, nn, bv);
  load4_row<Elem>(p.C, r * p.cs + n0, nn, cv);
  if (slot < 0 || slot >= p.nslots) {  // a row of no slot: zeros
    if (own) static_cast<Elem*>(p.out)[int64_t(r) * p.dim + mine] = Elem(0);
    return;
  }
  // (all of the states first: between loads of A, which many rows share, they take a fifth longer)
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int64_t ch = first_ch + k * CPW;
    load4<kStream>(p.state + (int64_t(slot) * p.dim + ch) * p.dstate + n0, ch < p.dim ? nn : 0, h[k]);
  }
  if constexpr (!kHeads) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int64_t ch = first_ch + k * CPW;
      load4<false>(p.A + ch * p.dstate + n0, ch < p.dim ? nn : 0, a[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[k][i] *= kLog2e;
    }
  }
  __shared__ int found[2][kWaves][2];
  int turn = 0;
  SlotOrder order[1] = {{true, INT32_MAX}};
  const int slots[1] = {slot};
  if (p.slots) slot_order<kWaves, 1>(p.slots, p.batch, r, slots, found, turn, order);
  if (!order[0].first) return;  // the first row of this slot takes this one
  for (;;) {
    float dt = c.dt + bias;
    if (p.softplus) dt = softplus_f(dt);
    const float dx = dt * c.x;
    const float deal = kHeads ? exp2_hw(dt * head_a) : dt;  // Mamba-2: the decay itself
    float y[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int from = k * CPW + (lane >> LG);
      const float dk = __shfl(deal, from, 64), dxk = __shfl(dx, from, 64);
      y[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float keep = kHeads ? dk : exp2_hw(dk * a[kHeads ? 0 : k][i]);
        h[k][i] = __builtin_fmaf(keep, h[k][i], dxk * bv[i]);
        // (a lane's states past dstate add nothing, whatever dt x is)
        y[k] = i < nn ? __builtin_fmaf(cv[i], h[k][i], y[k]) : y[k];
      }
    }
    float yc = 0.0f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const float v = __shfl(sum_lanes<LG>(y[k]), (lane & (CPW - 1)) << LG, 64);
      yc = (lane / CPW) == k ? v : yc;
    }
    if (own) {
      float v = p.D ? __builtin_fmaf(skip, c.x, yc) : yc;
      if (p.z) v = gate_f(v, c.z);
      static_cast<Elem*>(p.out)[int64_t(r) * p.dim + mine] = narrow<Elem>(v);
    }
    if (order[0].next == INT32_MAX) break;
    r = order[0].next;
    slot_order<kWaves, 1>(p.slots, p.batch, r, slots, found, turn ^= 1, order);
    c = load_channel(r);
    load4_row<Elem>(p.B, r * p.bs + n0, nn, bv);
    load4_row<Elem>(p.C, r * p.cs + n0, nn, cv);
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int64_t ch = first_ch + k * CPW;
    const int n = ch < p.dim ? nn : 0;
    store4<kStream>(p.state + (int64_t(slot) * p.dim + ch) * p.dstate + n0, n, h[k]);
  }
}

template <typename Elem, int LG, int CH, bool kStream>
void run_ch(const StepArgs& a, const StepParams& p, const StepForm& f, hipStream_t s) {
  const dim3 grid(unsigned(f.groups), unsigned(a.batch)), block(64 * kWaves);
  if (a.headdim)
    hipLaunchKernelGGL((state_step_kernel<Elem, LG, CH, true, kStream>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((state_step_kernel<Elem, LG, CH, false, kStream>), grid, block, 0, s, p);
}

template <typename Elem, int LG>
void run_lg(const StepArgs& a, const StepParams& p, hipStream_t s) {
  constexpr int most = step_most_channels(LG), few = step_few_channels(LG);
  const StepForm f = step_form(a.batch, a.dim, a.dstate);
  if (f.past_caches)
    run_ch<Elem, LG, most, true>(a, p, f, s);
  else if (f.channels == most)
    run_ch<Elem, LG, most, false>(a, p, f, s);
  else
    run_ch<Elem, LG, few, false>(a, p, f, s);
}

template <typename Elem>
void run(const StepArgs& a, const StepParams& p, hipStream_t s) {
  switch (step_lanes_log2(a.dstate)) {  // dstate <= 256, so at most 6
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
