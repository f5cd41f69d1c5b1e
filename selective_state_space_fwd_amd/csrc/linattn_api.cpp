// C-ABI entry points of linear attention (declared in include/ssm_linattn.h). Argument checking
// happens here, before any HIP call; the launches are in linattn_kernels.hip, linattn_bwd.hip
// and linattn_step.hip.
#include <stdint.h>

#include "api_util.h"
#include "heads.h"
#include "linattn_launch.h"
#include "ssm_linattn.h"

using ssm_api::aligned;
using ssm_api::check_heads;
using ssm_api::io_bytes;
using ssm_api::kInt32Max;
using ssm_api::product;
using ssm_api::Ranges;

namespace {

struct Sizes {
  int64_t batch, seqlen, qk_heads, heads, dk, dv;
  int64_t esz;
  int64_t state_bytes;  // of all rows and heads
  int64_t v_bytes, k_bytes;
};

ssm::Io io_of(int64_t esz) { return esz == 2 ? ssm::Io::BF16 : ssm::Io::F32; }

int check_sizes(uint32_t flags, uint32_t known, int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads,
                int64_t dk, int64_t dv, Sizes* z) {
  if (flags & ~(uint32_t(SSM_IO_MASK) | known)) return SSM_ERR_INVALID_ARG;
  if (batch < 0 || seqlen < 0 || qk_heads < 0 || heads < 0 || dk < 0 || dv < 0) return SSM_ERR_INVALID_ARG;
  if (heads > 0 && (qk_heads == 0 || heads % qk_heads != 0)) return SSM_ERR_INVALID_ARG;
  if (heads == 0 && qk_heads > 0) return SSM_ERR_INVALID_ARG;
  const int64_t esz = io_bytes(flags);
  if (esz == 0 || dk < 1 || dk > ssm::kLinattnMaxDim || dv < 1 || dv > ssm::kLinattnMaxDim || batch > 65535 ||
      seqlen > kInt32Max || heads > kInt32Max)
    return SSM_ERR_UNSUPPORTED;
  *z = Sizes{batch, seqlen, qk_heads, heads, dk, dv, esz, 0, 0, 0};
  z->state_bytes = product({batch, heads, dk, dv, 4});
  z->v_bytes = product({batch, seqlen, heads, dv, esz});
  z->k_bytes = product({batch, seqlen, qk_heads, dk, esz});
  if (z->state_bytes < 0 || z->v_bytes < 0 || z->k_bytes < 0 || product({batch, seqlen, heads, 4}) < 0)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// The strides of g (batch, step, head) and its bytes.
int check_gates(const float* g, const int64_t* strides, const Sizes& z, ssm::LinattnArgs* a, int64_t* bytes) {
  ssm::HeadRows rows;
  if (int st = check_heads(g, strides, z.batch, z.seqlen, z.heads, 1, 4, &rows, bytes)) return st;
  a->g = g;
  a->g_batch = rows.batch;
  a->g_step = rows.step;
  a->g_head = rows.head;
  if (!g) *bytes = 0;
  return SSM_OK;
}

bool grids_fit(const Sizes& z, bool bwd) {
  const ssm::Io io = io_of(z.esz);
  const int64_t c = ssm::linattn_bwd_chunk(io, z.dk, z.dv), chunks = (z.seqlen + c - 1) / c;
  const int64_t bh = product({z.batch, z.heads});
  if (bh < 0) return false;
  if (!bwd) {
    const ssm::LinattnSegments s = ssm::linattn_segments(z.batch, z.heads, z.dk, z.dv, z.seqlen, io);
    const int64_t blocks = ssm::linattn_join_blocks(ssm::linattn_state_floats(z.dv, z.dk));
    const int64_t a = product({bh, s.count, 4}), b = product({bh, blocks});
    return a >= 0 && b >= 0 && ssm::grid_fits(a, 256) && ssm::grid_fits(b, 256);
  }
  const int64_t blocks = ssm::linattn_join_blocks(ssm::linattn_state_floats(z.dk, z.dv));
  const int64_t a = product({bh, chunks, 8}), b = product({bh, blocks});
  return a >= 0 && b >= 0 && ssm::grid_fits(a, 256) && ssm::grid_fits(b, 256);
}

// The steps of every array, the results' among them.
bool steps_fit(const Sizes& z, const ssm::LinattnArgs& a) {
  for (int64_t step : {a.q.step, a.k.step, a.v.step, a.dout.step, z.heads * z.dv, z.qk_heads * z.dk})
    if (!ssm::linattn_reach(step, z.esz)) return false;
  return ssm::linattn_reach(a.g_step, 4);
}

int64_t fwd_workspace(const Sizes& z) {
  const ssm::LinattnSegments s = ssm::linattn_segments(z.batch, z.heads, z.dk, z.dv, z.seqlen, io_of(z.esz));
  if (s.count <= 1) return 0;
  return product({z.batch, z.heads, s.count, ssm::linattn_state_floats(z.dk, z.dv) + 1, 4});
}

int64_t bwd_workspace(const Sizes& z) {
  // (the sizes' products are known to fit: twice the states of every chunk)
  const int64_t c = ssm::linattn_bwd_chunk(io_of(z.esz), z.dk, z.dv), chunks = (z.seqlen + c - 1) / c;
  if (product({z.batch, z.heads, chunks, 4 * ssm::linattn_state_floats(z.dk, z.dv) + 4, 4}) < 0) return -1;
  return ssm::linattn_bwd_states(z.batch, z.heads, z.dk, z.dv, z.seqlen, io_of(z.esz)).total * 4;
}

}  // namespace

extern "C" {

int64_t ssm_linattn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads, int64_t dk, int64_t dv,
                                        uint32_t flags) {
  Sizes z;
  if (check_sizes(flags, SSM_LINATTN_HEAD_DG, batch, seqlen, heads, heads, dk, dv, &z) != SSM_OK || !grids_fit(z, false))
    return -1;
  return fwd_workspace(z);
}

int64_t ssm_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads, int64_t dk, int64_t dv,
                                        uint32_t flags) {
  Sizes z;
  if (check_sizes(flags, SSM_LINATTN_HEAD_DG, batch, seqlen, heads, heads, dk, dv, &z) != SSM_OK || !grids_fit(z, true))
    return -1;
  return bwd_workspace(z);
}

int ssm_linattn_fwd(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides, const void* v,
                    const int64_t* v_strides, const float* g, const int64_t* g_strides, const float* initial_state,
                    const int32_t* lengths, float scale, uint32_t flags, void* out, float* final_state,
                    void* workspace, int64_t workspace_bytes, int64_t batch, int64_t seqlen, int64_t qk_heads,
                    int64_t heads, int64_t dk, int64_t dv, void* stream) {
  Sizes z;
  if (int st = check_sizes(flags, 0, batch, seqlen, qk_heads, heads, dk, dv, &z)) return st;
  ssm::LinattnArgs a{};
  int64_t qb, kb, vb, gb;
  int st;
  if ((st = check_heads(q, q_strides, batch, seqlen, qk_heads, dk, z.esz, &a.q, &qb)) ||
      (st = check_heads(k, k_strides, batch, seqlen, qk_heads, dk, z.esz, &a.k, &kb)) ||
      (st = check_heads(v, v_strides, batch, seqlen, heads, dv, z.esz, &a.v, &vb)) ||
      (st = check_gates(g, g_strides, z, &a, &gb)))
    return st;
  if (!grids_fit(z, false) || !steps_fit(z, a)) return SSM_ERR_UNSUPPORTED;
  const int64_t need = fwd_workspace(z);
  if (need < 0) return SSM_ERR_UNSUPPORTED;
  if (z.v_bytes > 0 && (!q || !k || !v || !out)) return SSM_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(z.esz);
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(out, e) || !aligned(g, 4) ||
      !aligned(initial_state, 4) || !aligned(lengths, 4) || !aligned(final_state, 4) || !aligned(workspace, 256))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  r.add(q, qb, false);
  r.add(k, kb, false);
  r.add(v, vb, false);
  r.add(g, gb, false);
  r.add(initial_state, z.state_bytes, false);
  r.add(lengths, batch * 4, false);
  r.add(out, z.v_bytes, true);
  r.add(final_state, z.state_bytes, true);
  r.add(workspace, need, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || heads == 0 || (seqlen == 0 && !final_state)) return SSM_OK;
  a.initial = initial_state;
  a.lengths = lengths;
  a.out = out;
  a.final_state = final_state;
  a.workspace = static_cast<float*>(workspace);
  a.batch = batch, a.seqlen = seqlen, a.qk_heads = qk_heads, a.heads = heads, a.dk = dk, a.dv = dv;
  a.scale = scale;
  a.io = io_of(z.esz);
  return ssm::launch_linattn_fwd(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

int ssm_linattn_bwd(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides, const void* v,
                    const int64_t* v_strides, const void* dout, const int64_t* dout_strides, const float* g,
                    const int64_t* g_strides, const float* initial_state, const int32_t* lengths,
                    const float* dfinal, float scale, uint32_t flags, void* dq_out, void* dk_out, void* dv_out,
                    float* dg, float* dinitial, void* workspace, int64_t workspace_bytes, int64_t batch,
                    int64_t seqlen, int64_t qk_heads, int64_t heads, int64_t dk, int64_t dv, void* stream) {
  Sizes z;
  if (int st = check_sizes(flags, SSM_LINATTN_HEAD_DG, batch, seqlen, qk_heads, heads, dk, dv, &z)) return st;
  ssm::LinattnArgs a{};
  int64_t qb, kb, vb, ob, gb;
  int st;
  if ((st = check_heads(q, q_strides, batch, seqlen, qk_heads, dk, z.esz, &a.q, &qb)) ||
      (st = check_heads(k, k_strides, batch, seqlen, qk_heads, dk, z.esz, &a.k, &kb)) ||
      (st = check_heads(v, v_strides, batch, seqlen, heads, dv, z.esz, &a.v, &vb)) ||
      (st = check_heads(dout, dout_strides, batch, seqlen, heads, dv, z.esz, &a.dout, &ob)) ||
      (st = check_gates(g, g_strides, z, &a, &gb)))
    return st;
  if (!grids_fit(z, true) || !steps_fit(z, a)) return SSM_ERR_UNSUPPORTED;
  const int64_t need = bwd_workspace(z);
  if (need < 0) return SSM_ERR_UNSUPPORTED;
  if (z.v_bytes > 0 && (!q || !k || !v || !dout || !dq_out || !dk_out || !dv_out)) return SSM_ERR_INVALID_ARG;
  if (dg && !g) return SSM_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(z.esz);
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(dout, e) || !aligned(dq_out, e) ||
      !aligned(dk_out, e) || !aligned(dv_out, e) || !aligned(g, 4) || !aligned(initial_state, 4) ||
      !aligned(lengths, 4) || !aligned(dfinal, 4) || !aligned(dg, 4) || !aligned(dinitial, 4) ||
      !aligned(workspace, 256))
    return SSM_ERR_MISALIGNED;
  const bool per_head = (flags & SSM_LINATTN_HEAD_DG) != 0;
  Ranges r;
  r.add(q, qb, false);
  r.add(k, kb, false);
  r.add(v, vb, false);
  r.add(dout, ob, false);
  r.add(g, gb, false);
  r.add(initial_state, z.state_bytes, false);
  r.add(lengths, batch * 4, false);
  r.add(dfinal, z.state_bytes, false);
  r.add(dq_out, z.k_bytes, true);
  r.add(dk_out, z.k_bytes, true);
  r.add(dv_out, z.v_bytes, true);
  r.add(dg, per_head ? heads * 4 : batch * seqlen * heads * 4, true);
  r.add(dinitial, z.state_bytes, true);
  r.add(workspace, need, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (heads == 0 || (batch == 0 && !(dg && per_head))) return SSM_OK;
  a.initial = initial_state;
  a.lengths = lengths;
  a.dfinal = dfinal;
  a.dq = dq_out;
  a.dk_ = dk_out;
  a.dv_ = dv_out;
  a.dg = dg;
  a.dg_per_head = per_head;
  a.dinitial = dinitial;
  a.workspace = static_cast<float*>(workspace);
  a.batch = batch, a.seqlen = seqlen, a.qk_heads = qk_heads, a.heads = heads, a.dk = dk, a.dv = dv;
  a.scale = scale;
  a.io = io_of(z.esz);
  return ssm::launch_linattn_bwd(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

int ssm_linattn_step(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides, const void* v,
                     const int64_t* v_strides, const float* g, const int64_t* g_strides, const int32_t* slots,
                     float scale, uint32_t flags, float* state, void* out, int64_t batch, int64_t nslots,
                     int64_t qk_heads, int64_t heads, int64_t dk, int64_t dv, void* stream) {
  Sizes z;
  if (int st = check_sizes(flags, 0, batch, 1, qk_heads, heads, dk, dv, &z)) return st;
  if (nslots < 0 || (!slots && nslots < batch)) return SSM_ERR_INVALID_ARG;
  const int64_t cache = product({nslots, heads, dk, dv, 4});
  if (nslots > kInt32Max || cache < 0 ||
      !ssm::grid_fits(ssm::linattn_step_form(heads, dk, dv).groups, 64 * ssm::kLinattnStepWaves))
    return SSM_ERR_UNSUPPORTED;
  ssm::LinattnStepArgs a{};
  ssm::HeadRows gates;
  int64_t qb, kb, vb, gb, three[4][3];
  const int64_t* given[4] = {q_strides, k_strides, v_strides, g_strides};
  for (int i = 0; i < 4; ++i)
    if (given[i]) three[i][0] = given[i][0], three[i][1] = 0, three[i][2] = given[i][1];
  int st;
  if ((st = check_heads(q, q_strides ? three[0] : nullptr, batch, 1, qk_heads, dk, z.esz, &a.q, &qb)) ||
      (st = check_heads(k, k_strides ? three[1] : nullptr, batch, 1, qk_heads, dk, z.esz, &a.k, &kb)) ||
      (st = check_heads(v, v_strides ? three[2] : nullptr, batch, 1, heads, dv, z.esz, &a.v, &vb)) ||
      (st = check_heads(g, g_strides ? three[3] : nullptr, batch, 1, heads, 1, 4, &gates, &gb)))
    return st;
  if ((z.v_bytes > 0 && (!q || !k || !v || !out)) || (cache > 0 && !state)) return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(z.esz);
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(out, e) || !aligned(g, 4) ||
      !aligned(slots, 4) || !aligned(state, 4))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  r.add(q, qb, false);
  r.add(k, kb, false);
  r.add(v, vb, false);
  r.add(g, gb, false);
  r.add(slots, batch * 4, false);
  r.add(out, z.v_bytes, true);
  r.add(state, cache, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (batch == 0 || heads == 0) return SSM_OK;
  a.g = g;
  a.g_batch = gates.batch, a.g_head = gates.head;
  a.state = state, a.slots = slots, a.out = out;
  a.batch = batch, a.nslots = nslots, a.qk_heads = qk_heads, a.heads = heads, a.dk = dk, a.dv = dv;
  a.scale = scale;
  a.io = io_of(z.esz);
  return ssm::launch_linattn_step(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
