// One token of linear attention against a cache of states on gfx950 (include/ssm_linattn.h):
//
//   S = exp(g) S + v k^T;  out = scale S q
//
// The fp32 state is all of the traffic, read and written once, so the layout is the state's: a lane
// holds four consecutive k (16 bytes) of R rows v, the lanes of a row are consecutive and a power
// of two in number. q, k and the decay are the head's, the same for its rows; a row's v is loaded
// by one lane each and dealt out, and its result goes back the same way. A state is not read again
// before the next token, so it goes past L2 both ways: 32 heads of 128 x 64, b32 (67 MB moved) 18.9 ->
// 12.7 us, b64 32.7 -> 24.6, b128 57 -> 50, and no slower where one cache of 17 MB stays in the caches.
//
// Memory binds it: b512, 32 heads of 128 x 64 (1080 MB) 188 us, 5.7 TB/s (a copy's rate is 5.1); b8, 16 heads
// of 128 x 128 (17 MB) 5.9 us, where a launch is most of it.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_block.h"
#include "linattn_launch.h"

namespace ssm {
namespace {

constexpr int kWaves = kLinattnStepWaves;

struct LinattnStepParams {
  HeadRows q, k, v;
  const float* g;
  int64_t g_batch, g_head;
  float* state;
  const int32_t* slots;
  void* out;
  int64_t nslots;
  int batch, heads, group, dk, dv, tiles;
  float scale;
};

typedef float quad_t __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ void load_state(const float* p, int n, float (&v)[4]) {
  if (n >= 4) {
    const quad_t q = __builtin_nontemporal_load(reinterpret_cast<const quad_t*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = q[i];
  } else {
    load_part_of<float, 4>(p, n, v);
  }
}

// LG: log2 of the lanes of a row. R: rows a lane, at most as many as lanes of a row.
template <typename Elem, int LG, int R>
__global__ __launch_bounds__(64 * kWaves) void linattn_step_kernel(LinattnStepParams p) {
  constexpr int RPA = 64 >> LG;  // rows per access of a wave
  static_assert(R * RPA <= 64, "a lane for each row's v");
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tile = blockIdx.x % p.tiles, h = blockIdx.x / p.tiles, hk = h / p.group;
  int row = blockIdx.y;
  const int k0 = (lane & ((1 << LG) - 1)) * 4, nk = p.dk - k0 < 4 ? p.dk - k0 : 4;
  const int v0 = (tile * kWaves + wave) * (R * RPA);  // the wave's first row
  const int mine = v0 + lane;                         // the row whose v this lane loads
  const bool own = lane < R * RPA && mine < p.dv;
  const int slot = p.slots ? p.slots[row] : row;

  const Elem* qb = static_cast<const Elem*>(p.q.p) + hk * p.q.head + k0;
  const Elem* kb = static_cast<const Elem*>(p.k.p) + hk * p.k.head + k0;
  const Elem* vb = static_cast<const Elem*>(p.v.p) + h * p.v.head + mine;
  Elem* ob = static_cast<Elem*>(p.out) + int64_t(h) * p.dv + mine;
  const int64_t out_row = int64_t(p.heads) * p.dv;
  if (slot < 0 || slot >= p.nslots) {  // a row of no slot: zeros
    if (own) ob[row * out_row] = Elem(0);
    return;
  }
  float* state = p.state + (int64_t(slot) * p.heads + h) * p.dv * p.dk + k0;
  float s[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int v = v0 + i * RPA + (lane >> LG);
    load_state(state + int64_t(v) * p.dk, v < p.dv ? nk : 0, s[i]);
  }
  float q[4], k[4], v = 0.0f, g = 0.0f;
  auto load_token = [&] {
    load_part_of<Elem, 4>(qb + row * p.q.batch, nk, q);
    load_part_of<Elem, 4>(kb + row * p.k.batch, nk, k);
    v = own ? widen<Elem>(vb[row * p.v.batch]) : 0.0f;
    g = p.g ? p.g[row * p.g_batch + h * p.g_head] : 0.0f;
  };
  load_token();
  __shared__ int found[2][kWaves][2];
  int turn = 0;
  SlotOrder order[1] = {{true, INT32_MAX}};
  const int slots[1] = {slot};
  if (p.slots) slot_order<kWaves, 1>(p.slots, p.batch, row, slots, found, turn, order);
  if (!order[0].first) return;  // the first row of this slot takes this one
  for (;;) {
    const float keep = exp2_hw(g * kLog2e);
    float y[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float vi = __shfl(v, i * RPA + (lane >> LG), 64);
      y[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = __builtin_fmaf(keep, s[i][e], vi * k[e]);
        // (a lane's values past dk add nothing, whatever v is)
        y[i] = e < nk ? __builtin_fmaf(q[e], s[i][e], y[i]) : y[i];
      }
    }
    float mine_y = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float t = __shfl(sum_lanes<LG>(y[i]), (lane & (RPA - 1)) << LG, 64);
      mine_y = lane / RPA == i ? t : mine_y;
    }
    if (own) ob[row * out_row] = narrow<Elem>(p.scale * mine_y);
    if (order[0].next == INT32_MAX) break;
    row = order[0].next;
    slot_order<kWaves, 1>(p.slots, p.batch, row, slots, found, turn ^= 1, order);
    load_token();
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int vr = v0 + i * RPA + (lane >> LG);
    float* to = state + int64_t(vr) * p.dk;
    store_run_stream<float, 4>(to, vr < p.dv ? nk : 0, s[i]);
  }
}

template <typename Elem, int LG>
void run_lg(const LinattnStepParams& p, const LinattnStepForm& f, hipStream_t s) {
  constexpr int most = linattn_step_most_rows(LG), less = linattn_step_less_rows(LG);
  const dim3 grid(unsigned(f.groups), unsigned(p.batch)), block(64 * kWaves);
  if (f.rows == most)
    hipLaunchKernelGGL((linattn_step_kernel<Elem, LG, most>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((linattn_step_kernel<Elem, LG, less>), grid, block, 0, s, p);
}

template <typename Elem>
void run(const LinattnStepParams& p, const LinattnStepForm& f, hipStream_t s) {
  switch (step_lanes_log2(p.dk)) {  // dk <= 256, so at most 6
    case 0: return run_lg<Elem, 0>(p, f, s);
    case 1: return run_lg<Elem, 1>(p, f, s);
    case 2: return run_lg<Elem, 2>(p, f, s);
    case 3: return run_lg<Elem, 3>(p, f, s);
    case 4: return run_lg<Elem, 4>(p, f, s);
    case 5: return run_lg<Elem, 5>(p, f, s);
    default: return run_lg<Elem, 6>(p, f, s);
  }
}

}  // namespace

int launch_linattn_step(const LinattnStepArgs& a, void* stream) {
  const LinattnStepForm f = linattn_step_form(a.heads, a.dk, a.dv);
  LinattnStepParams p{};
  p.q = a.q, p.k = a.k, p.v = a.v;
  p.g = a.g, p.g_batch = a.g_batch, p.g_head = a.g_head;
  p.state = a.state, p.slots = a.slots, p.out = a.out, p.nslots = a.nslots;
  p.batch = int(a.batch), p.heads = int(a.heads), p.group = int(a.heads / a.qk_heads);
  p.dk = int(a.dk), p.dv = int(a.dv), p.tiles = int(f.tiles), p.scale = a.scale;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.io == Io::BF16)
    run<uint16_t>(p, f, s);
  else
    run<float>(p, f, s);
  return hipGetLastError() == hipSuccess ? 0 : -1;
}

}  // namespace ssm
