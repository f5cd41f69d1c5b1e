// C-ABI entry points of the gated RMS norm (declared in include/ssm_norm.h). Argument checking
// happens here, before any HIP call; the launches are in norm_kernels.hip.
#include <stdint.h>

#include <initializer_list>

#include "api_util.h"
#include "block_launch.h"
#include "ssm_norm.h"
#include "strided.h"

using ssm_api::aligned;
using ssm_api::check_strided;
using ssm_api::kInt32Max;
using ssm_api::mul_ok;
using ssm_api::Ranges;
using ssm_api::StridedArray;

namespace {

// Channels of a group that a workgroup always holds whole, in one step per lane (16 waves of
// 64 lanes of four fp32 channels).
constexpr int64_t kWholeChannels = int64_t(ssm::kNormMostWaves) * 64 * 4;

int check_sizes(uint32_t flags, int64_t batch, int64_t dim, int64_t groups, int64_t seqlen, int64_t* esz,
                int64_t* elems) {
  if (flags & ~uint32_t(SSM_IO_MASK | SSM_NORM_BEFORE_GATE)) return SSM_ERR_INVALID_ARG;
  if (batch < 0 || dim < 0 || seqlen < 0 || groups < 1 || dim % groups) return SSM_ERR_INVALID_ARG;
  const uint32_t io = flags & SSM_IO_MASK;
  if (io != SSM_IO_F32 && io != SSM_IO_BF16) return SSM_ERR_UNSUPPORTED;
  *esz = io == SSM_IO_BF16 ? 2 : 4;
  int64_t rows, bytes, tokens, groups_all;
  if (batch > kInt32Max || dim > kInt32Max || seqlen > kInt32Max || !mul_ok(batch, dim, &rows) ||
      !mul_ok(rows, seqlen, elems) || !mul_ok(*elems, 4, &bytes) || !mul_ok(batch, seqlen, &tokens) ||
      // at most one workgroup per token and group, or per token and block of 32 channels
      !mul_ok(tokens, groups + dim / 32, &groups_all) || groups_all > kInt32Max)
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Bytes of the blocks' sums of a split norm; -1 past int64.
int64_t split_bytes(int64_t batch, int64_t dim, int64_t groups, int64_t seqlen, ssm::Io io, int steps) {
  const int64_t blocks = ssm::norm_split_shape(dim / groups, seqlen, io, steps).cblocks;
  int64_t n;
  return mul_ok(batch * groups * seqlen, blocks * 4, &n) ? n : -1;
}

ssm::View view(const void* p, const StridedArray& a) { return ssm::View{p, a.s, a.order}; }

// One token per batch row and channels contiguous throughout: the batch is taken as the time
// axis, so that tokens share workgroups and partial sums.
bool one_token_rows(const ssm::NormArgs& a, const ssm::View* v, int n) {
  if (a.seqlen != 1 || a.batch == 1) return false;
  for (int i = 0; i < n; ++i)
    if (v[i].p && v[i].order != ssm::Order::Channel) return false;
  return true;
}

void batch_as_time(ssm::View* v) { v->s = ssm::Strides{0, v->s.channel, v->s.batch}; }

}  // namespace

extern "C" {

int64_t ssm_norm_fwd_workspace_bytes(int64_t batch, int64_t dim, int64_t groups, int64_t seqlen,
                                     uint32_t flags) {
  int64_t esz, elems;
  if (check_sizes(flags & SSM_IO_MASK, batch, dim, groups, seqlen, &esz, &elems) != SSM_OK) return -1;
  if (elems == 0) return 0;
  const ssm::Io io = esz == 2 ? ssm::Io::BF16 : ssm::Io::F32;
  return split_bytes(batch, dim, groups, seqlen, io, ssm::kNormFwdSteps[int(io)]);
}

int ssm_norm_fwd(const void* y, const int64_t* y_strides, const void* z, const int64_t* z_strides,
                 const float* weight, float eps, uint32_t flags, void* out, const int64_t* out_strides,
                 float* rstd, void* workspace, int64_t workspace_bytes, int64_t batch, int64_t dim,
                 int64_t groups, int64_t seqlen, void* stream) {
  int64_t esz, elems;
  if (int st = check_sizes(flags, batch, dim, groups, seqlen, &esz, &elems)) return st;
  if (!(eps >= 0.0f)) return SSM_ERR_INVALID_ARG;
  StridedArray ya, za, oa;
  if (int st = check_strided(y_strides, batch, dim, seqlen, esz, false, &ya)) return st;
  if (int st = z ? check_strided(z_strides, batch, dim, seqlen, esz, false, &za) : SSM_OK) return st;
  if (int st = check_strided(out_strides, batch, dim, seqlen, esz, true, &oa)) return st;
  if ((elems > 0 && (!y || !out)) || (dim > 0 && !weight)) return SSM_ERR_INVALID_ARG;
  // Where no split can come about, the workspace is not looked at.
  int64_t need = 0;
  const bool chan = ya.order == ssm::Order::Channel && (!z || za.order == ssm::Order::Channel) &&
                    oa.order == ssm::Order::Channel;
  if (elems > 0 && (!chan || dim / groups > kWholeChannels))
    need = ssm_norm_fwd_workspace_bytes(batch, dim, groups, seqlen, flags);
  if (need < 0) return SSM_ERR_UNSUPPORTED;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(esz);
  if (!aligned(y, e) || !aligned(z, e) || !aligned(out, e) || !aligned(weight, 4) || !aligned(rstd, 4) ||
      (need > 0 && !aligned(workspace, 256)))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  r.add(y, ya.bytes, false);
  r.add(z, za.bytes, false);
  r.add(weight, dim * 4, false);
  r.add(out, oa.bytes, true);
  r.add(rstd, elems > 0 ? batch * groups * seqlen * 4 : 0, true);
  r.add(workspace, need, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (elems == 0) return SSM_OK;
  ssm::NormArgs a{};
  a.batch = batch;
  a.dim = dim;
  a.groups = groups;
  a.seqlen = seqlen;
  a.weight = weight;
  a.rstd = rstd;
  a.rs = ssm::Strides{groups * seqlen, seqlen, 1};
  a.eps = eps;
  a.workspace = static_cast<float*>(workspace);
  a.io = esz == 2 ? ssm::Io::BF16 : ssm::Io::F32;
  a.norm_first = (flags & SSM_NORM_BEFORE_GATE) != 0;
  ssm::View v[3] = {view(y, ya), view(z, za), view(out, oa)};
  if (one_token_rows(a, v, 3)) {
    for (ssm::View& w : v) batch_as_time(&w);
    a.rs = ssm::Strides{0, 1, groups};
    a.seqlen = batch;
    a.batch = 1;
  }
  a.y = v[0];
  a.z = v[1];
  a.out = v[2];
  if (!ssm::norm_fits(a, ssm::norm_fwd_shape(a))) return SSM_ERR_UNSUPPORTED;
  return ssm::launch_norm_fwd(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

int64_t ssm_norm_bwd_workspace_bytes(int64_t batch, int64_t dim, int64_t groups, int64_t seqlen,
                                     uint32_t flags) {
  int64_t esz, elems, total;
  if (check_sizes(flags & SSM_IO_MASK, batch, dim, groups, seqlen, &esz, &elems) != SSM_OK) return -1;
  if (elems == 0) return 0;
  const ssm::Io io = esz == 2 ? ssm::Io::BF16 : ssm::Io::F32;
  // The most of any orders, and of a batch of single tokens taken as one sequence.
  const int64_t g = dim / groups, sums = split_bytes(batch, dim, groups, seqlen, io, ssm::kNormBwdSteps[int(io)]);
  const int steps = ssm::kNormBwdSteps[int(io)];
  int64_t n = 0;
  for (const ssm::NormShape& s : {ssm::norm_whole_shape(g, seqlen, io, steps, 8),
                                  ssm::norm_whole_shape(g, seqlen, io, steps, 16),
                                  ssm::norm_split_shape(g, seqlen, io, steps)})
    n = ssm::norm_partials(batch, s) > n ? ssm::norm_partials(batch, s) : n;
  if (sums < 0 || !mul_ok(n, dim * 4, &total) || total > INT64_MAX - sums) return -1;
  return total + sums;
}

int ssm_norm_bwd(const void* y, const int64_t* y_strides, const void* z, const int64_t* z_strides,
                 const float* weight, const float* rstd, const void* dout, const int64_t* dout_strides,
                 uint32_t flags, void* dy, const int64_t* dy_strides, void* dz, const int64_t* dz_strides,
                 float* dweight, void* workspace, int64_t workspace_bytes, int64_t batch, int64_t dim,
                 int64_t groups, int64_t seqlen, void* stream) {
  int64_t esz, elems;
  if (int st = check_sizes(flags, batch, dim, groups, seqlen, &esz, &elems)) return st;
  StridedArray ya, za, ga, dya, dza;
  if (int st = check_strided(y_strides, batch, dim, seqlen, esz, false, &ya)) return st;
  if (int st = z ? check_strided(z_strides, batch, dim, seqlen, esz, false, &za) : SSM_OK) return st;
  if (int st = check_strided(dout_strides, batch, dim, seqlen, esz, false, &ga)) return st;
  if (int st = check_strided(dy_strides, batch, dim, seqlen, esz, true, &dya)) return st;
  if (int st = z ? check_strided(dz_strides, batch, dim, seqlen, esz, true, &dza) : SSM_OK) return st;
  const int64_t need = ssm_norm_bwd_workspace_bytes(batch, dim, groups, seqlen, flags);
  if (need < 0) return SSM_ERR_UNSUPPORTED;
  if ((elems > 0 && (!y || !rstd || !dout || !dy || (z && !dz))) || (dim > 0 && (!weight || !dweight)))
    return SSM_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(esz);
  if (!aligned(y, e) || !aligned(z, e) || !aligned(dout, e) || !aligned(dy, e) || (z && !aligned(dz, e)) ||
      !aligned(weight, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(workspace, 256))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  r.add(y, ya.bytes, false);
  r.add(z, za.bytes, false);
  r.add(weight, dim * 4, false);
  r.add(rstd, elems > 0 ? batch * groups * seqlen * 4 : 0, false);
  r.add(dout, ga.bytes, false);
  r.add(dy, dya.bytes, true);
  if (z) r.add(dz, dza.bytes, true);
  r.add(dweight, dim * 4, true);
  r.add(workspace, need, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (dim == 0) return SSM_OK;
  ssm::NormArgs a{};
  a.batch = batch;
  a.dim = dim;
  a.groups = groups;
  a.seqlen = seqlen;
  a.weight = weight;
  a.rstd = const_cast<float*>(rstd);
  a.rs = ssm::Strides{groups * seqlen, seqlen, 1};
  a.dweight = dweight;
  a.workspace = static_cast<float*>(workspace);
  a.io = esz == 2 ? ssm::Io::BF16 : ssm::Io::F32;
  a.norm_first = (flags & SSM_NORM_BEFORE_GATE) != 0;
  ssm::View v[5] = {view(y, ya), view(z, za), view(dout, ga), view(dy, dya), view(z ? dz : nullptr, dza)};
  if (one_token_rows(a, v, 5)) {
    for (ssm::View& w : v) batch_as_time(&w);
    a.rs = ssm::Strides{0, 1, groups};
    a.seqlen = batch;
    a.batch = 1;
  }
  a.y = v[0];
  a.z = v[1];
  a.dout = v[2];
  a.dy = v[3];
  a.dz = v[4];
  if ((elems > 0 && !ssm::norm_fits(a, ssm::norm_bwd_shape(a))) ||
      !ssm::grid_fits(ssm::reduce_groups(dim), ssm::kReduceCols * ssm::kNormReduceSlices))
    return SSM_ERR_UNSUPPORTED;
  return ssm::launch_norm_bwd(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
