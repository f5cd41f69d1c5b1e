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

// Heads of one step that a row's lanes take one after another, all loads first: they share the
// angles. One where the call is small, for more waves.
constexpr int kQkMostRows = 4;
inline int qk_rows(int64_t batch, int64_t seqlen, int64_t heads, int lg) {
  return ((batch * seqlen * heads) >> (6 - lg)) / kQkMostRows >= 4096 ? kQkMostRows : 1;
}

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

// Workgroups of a side in the backward, each with one row of partial weight gradients.
constexpr int64_t kQkMostPartials = 2048;
inline int64_t qk_partials(int64_t groups) { return groups < kQkMostPartials ? groups : kQkMostPartials; }

int launch_qk_fwd(const QkArgs& a, void* stream);
int launch_qk_bwd(const QkArgs& a, void* stream);

}  // namespace ssm
