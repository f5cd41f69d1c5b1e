// C-ABI entry points of the norm and rotation of queries and keys (declared in include/ssm_qk.h).
// Argument checking happens here, before any HIP call; the launches are in qk_kernels.hip.
#include <stdint.h>

#include "api_util.h"
#include "heads.h"
#include "qk_launch.h"
#include "ssm_qk.h"

using ssm_api::aligned;
using ssm_api::check_heads;
using ssm_api::io_bytes;
using ssm_api::kInt32Max;
using ssm_api::product;
using ssm_api::Ranges;

namespace {

struct Sizes {
  int64_t esz, q_bytes, k_bytes, table_bytes, workspace;
};

int check_sizes(uint32_t flags, int64_t batch, int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim,
                int64_t rot, int64_t table_rows, Sizes* z) {
  if (flags & ~(uint32_t(SSM_IO_MASK) | SSM_QK_INTERLEAVED)) return SSM_ERR_INVALID_ARG;
  if (batch < 0 || seqlen < 0 || q_heads < 0 || k_heads < 0 || dim < 0 || rot < 0 || table_rows < 0)
    return SSM_ERR_INVALID_ARG;
  z->esz = io_bytes(flags);
  if (z->esz == 0 || dim < 1 || dim > ssm::kQkMaxDim || rot > dim || rot % 2 != 0 || q_heads > kInt32Max ||
      k_heads > kInt32Max - q_heads)
    return SSM_ERR_UNSUPPORTED;
  z->q_bytes = product({batch, seqlen, q_heads, dim, z->esz});
  z->k_bytes = product({batch, seqlen, k_heads, dim, z->esz});
  z->table_bytes = product({table_rows, rot / 2, 4});
  const int64_t steps = product({batch, seqlen, 4}), rows = product({batch, seqlen, q_heads + k_heads});
  if (z->q_bytes < 0 || z->k_bytes < 0 || z->table_bytes < 0 || steps < 0 || rows < 0) return SSM_ERR_UNSUPPORTED;
  const int lg = ssm::qk_lanes_log2(dim, rot);
  // The backward's items, no fewer than the forward's.
  const bool many = ssm::qk_many(batch, seqlen, q_heads + k_heads, lg);
  const int per = many ? ssm::qk_most_rows(true, int(z->esz)) : 1;
  const int64_t q_items = ssm::qk_items(batch, seqlen, q_heads, per), k_items = ssm::qk_items(batch, seqlen, k_heads, per);
  if (seqlen > kInt32Max || q_items > ssm::kQkMostItems || k_items > ssm::kQkMostItems) return SSM_ERR_UNSUPPORTED;
  const int64_t q_groups = ssm::qk_groups(q_items, lg), k_groups = ssm::qk_groups(k_items, lg);
  z->workspace = (ssm::qk_partials(q_groups, k_groups) + ssm::qk_partials(k_groups, q_groups)) * dim * 4;
  return ssm::grid_fits(q_groups + k_groups, 64 * ssm::kQkWaves) ? SSM_OK : SSM_ERR_UNSUPPORTED;
}

ssm::QkArgs common(const ssm::HeadRows& q, const ssm::HeadRows& k, const float* q_weight, const float* k_weight,
                   const float* cos, const float* sin, const int32_t* positions, float eps, uint32_t flags,
                   int64_t batch, int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim, int64_t rot,
                   int64_t table_rows) {
  ssm::QkArgs a{};
  a.q = q, a.k = k;
  a.q_weight = q_weight, a.k_weight = k_weight;
  a.cos = cos, a.sin = sin;
  a.positions = positions;
  a.eps = eps;
  a.interleaved = (flags & SSM_QK_INTERLEAVED) != 0;
  a.batch = batch, a.seqlen = seqlen, a.q_heads = q_heads, a.k_heads = k_heads;
  a.dim = dim, a.rot = rot, a.table_rows = table_rows;
  a.io = io_bytes(flags) == 2 ? ssm::Io::BF16 : ssm::Io::F32;
  return a;
}

}  // namespace

extern "C" {

int ssm_qk_norm_fwd(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                    const float* q_weight, const float* k_weight, const float* cos, const float* sin,
                    const int32_t* positions, float eps, uint32_t flags, void* q_out, void* k_out, int64_t batch,
                    int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim, int64_t rot, int64_t table_rows,
                    void* stream) {
  Sizes z;
  if (int st = check_sizes(flags, batch, seqlen, q_heads, k_heads, dim, rot, table_rows, &z)) return st;
  ssm::HeadRows qr, kr;
  int64_t qb, kb;
  int st;
  if ((st = check_heads(q, q_strides, batch, seqlen, q_heads, dim, z.esz, &qr, &qb)) ||
      (st = check_heads(k, k_strides, batch, seqlen, k_heads, dim, z.esz, &kr, &kb)))
    return st;
  if ((qb > 0 && (!q || !q_out)) || (kb > 0 && (!k || !k_out)) || (z.table_bytes > 0 && (!cos || !sin)))
    return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(z.esz);
  if (!aligned(q, e) || !aligned(k, e) || !aligned(q_out, e) || !aligned(k_out, e) || !aligned(q_weight, 4) ||
      !aligned(k_weight, 4) || !aligned(cos, 4) || !aligned(sin, 4) || !aligned(positions, 4))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  r.add(q, qb, false);
  r.add(k, kb, false);
  r.add(q_weight, dim * 4, false);
  r.add(k_weight, dim * 4, false);
  r.add(cos, z.table_bytes, false);
  r.add(sin, z.table_bytes, false);
  r.add(positions, batch * seqlen * 4, false);
  r.add(q_out, z.q_bytes, true);
  r.add(k_out, z.k_bytes, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (qb == 0 && kb == 0) return SSM_OK;
  ssm::QkArgs a = common(qr, kr, q_weight, k_weight, cos, sin, positions, eps, flags, batch, seqlen, q_heads,
                         k_heads, dim, rot, table_rows);
  a.q_out = q_out;
  a.k_out = k_out;
  return ssm::launch_qk_fwd(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

int64_t ssm_qk_norm_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim,
                                        int64_t rot, uint32_t flags) {
  Sizes z;
  if (check_sizes(flags, batch, seqlen, q_heads, k_heads, dim, rot, 0, &z) != SSM_OK) return -1;
  return z.workspace;
}

int ssm_qk_norm_bwd(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                    const void* dq_out, const int64_t* dq_out_strides, const void* dk_out,
                    const int64_t* dk_out_strides, const float* q_weight, const float* k_weight, const float* cos,
                    const float* sin, const int32_t* positions, float eps, uint32_t flags, void* dq, void* dk,
                    float* dq_weight, float* dk_weight, void* workspace, int64_t workspace_bytes, int64_t batch,
                    int64_t seqlen, int64_t q_heads, int64_t k_heads, int64_t dim, int64_t rot, int64_t table_rows,
                    void* stream) {
  Sizes z;
  if (int st = check_sizes(flags, batch, seqlen, q_heads, k_heads, dim, rot, table_rows, &z)) return st;
  ssm::HeadRows qr, kr, dqr, dkr;
  int64_t qb, kb, dqb, dkb;
  int st;
  if ((st = check_heads(q, q_strides, batch, seqlen, q_heads, dim, z.esz, &qr, &qb)) ||
      (st = check_heads(k, k_strides, batch, seqlen, k_heads, dim, z.esz, &kr, &kb)) ||
      (st = check_heads(dq_out, dq_out_strides, batch, seqlen, q_heads, dim, z.esz, &dqr, &dqb)) ||
      (st = check_heads(dk_out, dk_out_strides, batch, seqlen, k_heads, dim, z.esz, &dkr, &dkb)))
    return st;
  const bool sums = dq_weight || dk_weight;
  const int64_t need = sums ? z.workspace : 0;
  if ((qb > 0 && (!q || !dq_out || !dq)) || (kb > 0 && (!k || !dk_out || !dk)) ||
      (z.table_bytes > 0 && (!cos || !sin)) || (need > 0 && (!workspace || workspace_bytes < need)))
    return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(z.esz);
  if (!aligned(q, e) || !aligned(k, e) || !aligned(dq_out, e) || !aligned(dk_out, e) || !aligned(dq, e) ||
      !aligned(dk, e) || !aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(cos, 4) || !aligned(sin, 4) ||
      !aligned(positions, 4) || !aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(workspace, 256))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  r.add(q, qb, false);
  r.add(k, kb, false);
  r.add(dq_out, dqb, false);
  r.add(dk_out, dkb, false);
  r.add(q_weight, dim * 4, false);
  r.add(k_weight, dim * 4, false);
  r.add(cos, z.table_bytes, false);
  r.add(sin, z.table_bytes, false);
  r.add(positions, batch * seqlen * 4, false);
  r.add(dq, z.q_bytes, true);
  r.add(dk, z.k_bytes, true);
  r.add(dq_weight, dim * 4, true);
  r.add(dk_weight, dim * 4, true);
  r.add(workspace, need, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (qb == 0 && kb == 0 && !sums) return SSM_OK;
  ssm::QkArgs a = common(qr, kr, q_weight, k_weight, cos, sin, positions, eps, flags, batch, seqlen, q_heads,
                         k_heads, dim, rot, table_rows);
  a.dyq = dqr, a.dyk = dkr;
  a.q_out = dq, a.k_out = dk;
  a.dq_weight = dq_weight, a.dk_weight = dk_weight;
  a.workspace = static_cast<float*>(workspace);
  return ssm::launch_qk_bwd(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
