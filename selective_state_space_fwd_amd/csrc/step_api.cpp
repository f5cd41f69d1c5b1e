// C-ABI entry points of the single-token state update (declared in include/ssm_step.h).
// Argument checking happens here, before any HIP call; the launch is in step_kernels.hip.
#include <stdint.h>

#include "api_util.h"
#include "block_launch.h"
#include "ssm_step.h"
#include "strided.h"

using ssm_api::aligned;
using ssm_api::kInt32Max;
using ssm_api::mul_ok;
using ssm_api::Ranges;

namespace {

// Bytes from the first element of `rows` rows of `cols`, `stride` apart, to past the last.
int rows_bytes(int64_t rows, int64_t cols, int64_t stride, int64_t esz, int64_t* bytes) {
  *bytes = 0;
  if (rows == 0 || cols == 0) return SSM_OK;
  if (rows > 1 && stride < 0) return SSM_ERR_INVALID_ARG;
  int64_t reach;
  if (!mul_ok(rows - 1, rows > 1 ? stride : 0, &reach) || reach > INT64_MAX - cols ||
      !mul_ok(reach + cols, esz, bytes))
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Mamba-2 (heads of headdim channels) or Mamba-1 (headdim 0: `heads` channels).
int step_impl(const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, const float* A,
              const void* B, int64_t b_stride, const void* C, int64_t c_stride, const float* D,
              const void* z, int64_t z_stride, const float* dt_bias, const int32_t* slots, uint32_t flags,
              float* state, void* out, int64_t batch, int64_t nslots, int64_t heads, int64_t headdim,
              bool per_head, int64_t dstate, void* stream) {
  if (flags & ~uint32_t(SSM_IO_MASK | SSM_DELTA_SOFTPLUS)) return SSM_ERR_INVALID_ARG;
  if (batch < 0 || nslots < 0 || heads < 0 || headdim < 0 || dstate < 0) return SSM_ERR_INVALID_ARG;
  if (!slots && nslots < batch) return SSM_ERR_INVALID_ARG;
  const uint32_t io = flags & SSM_IO_MASK;
  if (io != SSM_IO_F32 && io != SSM_IO_BF16) return SSM_ERR_UNSUPPORTED;
  if (dstate < 1 || dstate > ssm::kStepMaxState) return SSM_ERR_UNSUPPORTED;
  if (per_head && headdim < 1) return SSM_ERR_UNSUPPORTED;
  const int64_t esz = io == SSM_IO_BF16 ? 2 : 4;
  int64_t dim, cache, cache_bytes, xb, tb, bb, cb, zb;
  if (!mul_ok(heads, per_head ? headdim : 1, &dim) || dim > kInt32Max || batch > 65535 ||
      nslots > kInt32Max || !mul_ok(nslots, dim, &cache) || !mul_ok(cache, dstate * 4, &cache_bytes) ||
      !ssm::grid_fits(ssm::step_form(batch, dim, dstate).groups, 64 * ssm::kStepWaves))
    return SSM_ERR_UNSUPPORTED;
  int st;
  if ((st = rows_bytes(batch, dim, x_stride, esz, &xb)) || (st = rows_bytes(batch, heads, dt_stride, esz, &tb)) ||
      (st = rows_bytes(batch, dstate, b_stride, esz, &bb)) ||
      (st = rows_bytes(batch, dstate, c_stride, esz, &cb)) ||
      (st = z ? rows_bytes(batch, dim, z_stride, esz, &zb) : (zb = 0, SSM_OK)))
    return st;
  const bool any = batch > 0 && dim > 0;
  if ((any && (!x || !dt || !B || !C || !out)) || (dim > 0 && !A) || (cache > 0 && !state))
    return SSM_ERR_INVALID_ARG;
  const uintptr_t e = uintptr_t(esz);
  if (!aligned(x, e) || !aligned(dt, e) || !aligned(B, e) || !aligned(C, e) || !aligned(z, e) ||
      !aligned(out, e) || !aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(slots, 4) ||
      !aligned(state, 4))
    return SSM_ERR_MISALIGNED;
  Ranges r;
  r.add(x, xb, false);
  r.add(dt, tb, false);
  r.add(A, (per_head ? heads : dim * dstate) * 4, false);
  r.add(B, bb, false);
  r.add(C, cb, false);
  r.add(D, dim * 4, false);
  r.add(z, zb, false);
  r.add(dt_bias, heads * 4, false);
  r.add(slots, batch * 4, false);
  r.add(out, batch * dim * esz, true);
  r.add(state, cache_bytes, true);
  if (r.clash()) return SSM_ERR_INVALID_ARG;
  if (!any) return SSM_OK;
  ssm::StepArgs a{x, dt, B, C, z, x_stride, dt_stride, b_stride, c_stride, z_stride, A, D, dt_bias, state,
                  slots, out, batch, nslots, dim, dstate, per_head ? headdim : 0,
                  io == SSM_IO_BF16 ? ssm::Io::BF16 : ssm::Io::F32, (flags & SSM_DELTA_SOFTPLUS) != 0};
  return ssm::launch_state_step(a, stream) == 0 ? SSM_OK : SSM_ERR_HIP;
}

}  // namespace

extern "C" {

int ssm_scan_step(const void* u, int64_t u_stride, const void* delta, int64_t delta_stride, const float* A,
                  const void* B, int64_t b_stride, const void* C, int64_t c_stride, const float* D,
                  const void* z, int64_t z_stride, const float* delta_bias, const int32_t* slots,
                  uint32_t flags, float* state, void* out, int64_t batch, int64_t nslots, int64_t dim,
                  int64_t dstate, void* stream) {
  return step_impl(u, u_stride, delta, delta_stride, A, B, b_stride, C, c_stride, D, z, z_stride, delta_bias,
                   slots, flags, state, out, batch, nslots, dim, 0, false, dstate, stream);
}

int ssm_ssd_step(const void* x, int64_t x_stride, const void* dt, int64_t dt_stride, const float* A,
                 const void* B, int64_t b_stride, const void* C, int64_t c_stride, const float* D, const void* z,
                 int64_t z_stride, const float* dt_bias, const int32_t* slots, uint32_t flags, float* state,
                 void* out, int64_t batch, int64_t nslots, int64_t nheads, int64_t headdim, int64_t dstate,
                 void* stream) {
  return step_impl(x, x_stride, dt, dt_stride, A, B, b_stride, C, c_stride, D, z, z_stride, dt_bias, slots,
                   flags, state, out, batch, nslots, nheads, headdim, true, dstate, stream);
}

}  // extern "C"
