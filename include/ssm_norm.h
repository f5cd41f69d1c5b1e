/*
 * ssm_norm.h -- C ABI of the gated RMS norm in libssmscan.so (gfx950): the norm over channels
 * between a Mamba block's scan and its output projection, with the gate on either side of it,
 * and its gradient. (The channel-wise normalisation that mhpq.cn/news/1057127, section 2, puts
 * beside the scan.)
 *
 * dim channels in `groups` equal groups of G; per token (batch row b, step t) and group, with
 * s = z * sigmoid(z) (1 without a gate):
 *
 *   out = weight * (y s) * r,    r = 1 / sqrt(mean_G((y s)^2) + eps)
 *   out = weight * y * r * s,    r = 1 / sqrt(mean_G(y^2) + eps)       (SSM_NORM_BEFORE_GATE)
 *
 * Memory: device pointers owned by the caller.
 *   y, z, out, dout, dy, dz : [batch, dim, seqlen] in the storage type, each with its own element
 *            strides {batch, channel, step} in a HOST array of three (NULL: contiguous); either
 *            the step or the channel stride is 1. So y can be the scan's output (steps
 *            contiguous), z a slice of a projection's (channels contiguous) and out what the
 *            next projection reads. Strides of inputs are >= 0; an output's must name every
 *            element once.
 *   weight, dweight : [dim] fp32
 *   rstd     : [batch, groups, seqlen] fp32, r of every token and group
 * Sums are fp32; results are rounded to the storage type once. The squares are fp32 too: a token
 * whose mean square (plus eps) is no normal fp32 number, values below some 1e-18 with eps 0 or
 * above 1e18, has no r. Calls are asynchronous on
 * `stream`, use no atomics (bitwise reproducible) and allocate nothing; every check happens
 * before any HIP call. Outputs must overlap no other argument (a strided array counts with its
 * whole extent). Returns SSM_OK, SSM_ERR_INVALID_ARG, SSM_ERR_UNSUPPORTED (a storage type other
 * than fp32/bf16, neither stride 1, dim or seqlen above 2^31 - 1, tokens times groups and
 * 32-channel blocks above 2^31 - 1, or more than a grid of 2^32 - 1 work-items takes: some 2^34
 * elements, less where groups of few channels meet sequences of few steps; a gradient of 2^27
 * channels), SSM_ERR_MISALIGNED (a pointer not aligned to its element size) or SSM_ERR_HIP.
 */
#ifndef SSM_NORM_H
#define SSM_NORM_H

#include <stdint.h>

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* flags: the storage type (SSM_IO_F32 or SSM_IO_BF16), and */
#define SSM_NORM_BEFORE_GATE (1u << 12)

/*
 * ssm_norm_fwd -- required: y, weight, out (NULL only when empty); optional (NULL): z (no
 * gate), rstd (not returned; the backward needs it). batch, dim, seqlen >= 0; groups >= 1 and a
 * divisor of dim; eps >= 0. workspace: ssm_norm_fwd_workspace_bytes(batch, dim, groups, seqlen,
 * flags) bytes (workspace_bytes, at least that), 256-byte aligned, overwritten; calls that share
 * it must not overlap in time. Not looked at (NULL) where every tensor has channel stride 1 and
 * a group at most 4096 channels; SSM_ERR_INVALID_ARG without it elsewhere.
 */
SSM_API int ssm_norm_fwd(const void* y, const int64_t* y_strides, const void* z,
                         const int64_t* z_strides, const float* weight, float eps,
                         uint32_t flags, void* out, const int64_t* out_strides, float* rstd,
                         void* workspace, int64_t workspace_bytes, int64_t batch, int64_t dim,
                         int64_t groups, int64_t seqlen, void* stream);

/* Bytes of workspace ssm_norm_fwd needs at most: a sum per token and block of channels. -1 as
 * ssm_norm_bwd_workspace_bytes. */
SSM_API int64_t ssm_norm_fwd_workspace_bytes(int64_t batch, int64_t dim, int64_t groups,
                                             int64_t seqlen, uint32_t flags);

/*
 * ssm_norm_bwd -- gradients of L = sum(dout * out): dy, dz (required when z is given),
 * dweight, overwritten. rstd: the forward's. workspace:
 * ssm_norm_bwd_workspace_bytes(batch, dim, groups, seqlen, flags) bytes (workspace_bytes, at
 * least that), 256-byte aligned, overwritten; calls that share it must not overlap in time.
 * dweight's sum over tokens is added in a fixed order.
 */
SSM_API int ssm_norm_bwd(const void* y, const int64_t* y_strides, const void* z,
                         const int64_t* z_strides, const float* weight, const float* rstd,
                         const void* dout, const int64_t* dout_strides, uint32_t flags,
                         void* dy, const int64_t* dy_strides, void* dz,
                         const int64_t* dz_strides, float* dweight, void* workspace,
                         int64_t workspace_bytes, int64_t batch, int64_t dim, int64_t groups,
                         int64_t seqlen, void* stream);

/* Bytes of workspace ssm_norm_bwd needs, whatever the strides: a partial sum of dweight per run
 * of tokens and a sum per token and block of channels. -1 for negative sizes, groups not a divisor of dim, an unknown storage type or a
 * size past int64. */
SSM_API int64_t ssm_norm_bwd_workspace_bytes(int64_t batch, int64_t dim, int64_t groups,
                                             int64_t seqlen, uint32_t flags);

#ifdef __cplusplus
}
#endif

#endif /* SSM_NORM_H */
