// Internal interface between the C-ABI layer of the queries' and keys' norm (qk_api.cpp) and its
// kernels. Not installed; the public ABI is include/ssm_qk.h.
#pragma once
#include <stdint.h>

#include "linattn_launch.h"

namespace ssm {

constexpr int kQkMaxDim = 256;
constexpr int kQkWaves = 4;

struct QkArgs {
  HeadRows q, k;             // [batch, seqlen, heads, dim]
  HeadRows dyq, dyk;         // backward: of the results
  const float *q_weight, *k_weight;  // nullable: [dim]
  const float *cos, *sin;    // [table_rows, rot / 2]; null where rot is 0
  const int32_t* positions;  // nullable: [batch, seqlen]
  float eps;
  bool interleaved;
  void *q_out, *k_out;       // contiguous: results, or dq and dk
  float *dq_weight, *dk_weight;  // nullable
  float* workspace;          // backward: qk_partials(...) rows of 2 dim floats
  int64_t batch, seqlen, q_heads, k_heads, dim, rot, table_rows;
  Io io;
};

// A lane's share of a row is eight values: four pairs that turn by four angles, or eight that do not
// turn. The lanes of a row, a power of two, 4 at least.
inline int qk_units(int64_t dim, int64_t rot) { return int((rot / 2 + 3) / 4 + (dim - rot + 7) / 8); }
inline int qk_lanes_log2(int64_t dim, int64_t rot) {
  int lg = 2;
  while ((1 << lg) < qk_units(dim, rot)) ++lg;
  return lg;
}

// Large calls, by the waves that hold one head a group of lanes: several heads a group, and results
// stored past L2. 32 + 8 heads of 128 in bf16, few | many, us (forward, gradient): 512 steps 5.2 12.1 |
// 5.5 10.5; 1024 steps (10240 waves) 7.9 15.2 | 6.5 13.7; 2048 steps 11.3 21.2 | 8.6 18.3; 8192 steps
// 38.9 64.5 | 32.1 53.0. fp32: 1024 steps 11.0 17.4 | 9.7 16.9; 8192 steps 62.7 84.3 | 57.8 81.5. Below, where both
// are near a launch, the results stay in L2 for what reads them next.
constexpr int64_t kQkManyWaves = 10240;
inline bool qk_many(int64_t batch, int64_t seqlen, int64_t heads, int lg) {
  return (batch * seqlen * heads) >> (6 - lg) >= kQkManyWaves;
}

// Heads of one step that a group of lanes takes together in a large call, all loads first: they share
// the angles. (bf16, 8192 steps of 32 + 8 heads of 128: forward 4 heads 32.1 us, 2 heads 33.7;
// gradient, its loads an item ahead, 4 heads 76.5 (spills), 2 heads 68.5, 1 head 75.2. fp32's two
// heads spill.)
constexpr int qk_most_rows(bool bwd, int bytes) { return bwd ? (bytes == 2 ? 2 : 1) : 4; }

// What one group of lanes takes: `rows` heads of one side (q or k) at one step; and the workgroups
// of a side.
inline int64_t qk_items(int64_t batch, int64_t seqlen, int64_t heads, int rows) {
  return batch * seqlen * ((heads + rows - 1) / rows);
}
inline int64_t qk_groups(int64_t items, int lg) {
  const int64_t per = int64_t(kQkWaves) << (6 - lg);
  return (items + per - 1) / per;
}
// Items are numbered in 32 bits.
constexpr int64_t kQkMostItems = (int64_t(1) << 31) - 1;

// Workgroups of a side in the backward, each with one row of partial weight gradients: no more than
// the chip holds at once, four a compute unit, shared between the sides by their items, each loading
// its next item while it works on this one. (bf16, 8192 steps of 32 + 8 heads of 128, five a compute
// unit: 1280 workgroups 71.1 us, 2560 78.6; four: 1024 68.5.)
constexpr int64_t kQkMostPartials = 1024;
inline int64_t qk_partials(int64_t groups, int64_t other) {
  const int64_t all = groups + other;
  return all <= kQkMostPartials ? groups : groups == 0 ? 0 : (kQkMostPartials * groups + all - 1) / all;
}

int launch_qk_fwd(const QkArgs& a, void* stream);
int launch_qk_bwd(const QkArgs& a, void* stream);

}  // namespace ssm
