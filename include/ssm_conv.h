/*
 * ssm_conv.h -- C ABI of the short causal convolution in libssmscan.so (gfx950): the
 * depthwise convolution over a few past steps that a Mamba block applies to the scan's input
 * (and Mamba-2 to B and C too), its gradient, and its single-token step against a cache of
 * request states (the conv_state of ybb.press/ai-applications/14118.html, section 5.1).
 *
 * For batch row b, channel d, step t and width W (2, 3 or 4):
 *
 *   p[b,d,t]   = bias[d] + sum_{k<W} weight[d,k] * x[b,d,t - (W-1) + k]    (bias optional)
 *   out[b,d,t] = p, or p * sigmoid(p) with SSM_CONV_SILU
 *
 * where the W-1 steps before the first are initial_state[b,d,0..W-2] (oldest first; zero if
 * NULL). With lengths, row b ends at step n = lengths[b] (clamped to [0, seqlen]): x at and
 * behind it is not read, out there is 0, and final_state[b,d,:], the last W-1 inputs, is taken
 * before it (from initial_state where the row is shorter). The scan's padding mask of the same
 * batch is t < lengths[b].
 *
 * Memory: device pointers owned by the caller.
 *   x, dx           : [batch, dim, seqlen] in the storage type, with element strides {batch,
 *                     channel, step} in a HOST array of three (NULL: contiguous); either the
 *                     step or the channel stride is 1 (a projection's output, token by token,
 *                     has channel stride 1 and needs no copy). Strides of inputs are >= 0;
 *                     dx's must name every element once and have x's
 *                     contiguous axis.
 *   out, dout       : [batch, dim, seqlen] contiguous, storage type
 *   initial_state, final_state, dfinal, dinitial : [batch, dim, W-1] contiguous, storage type
 *   weight, dweight : [dim, W]  fp32;  bias, dbias : [dim] fp32
 *   lengths         : [batch] int32
 * Sums are fp32; results are rounded to the storage type once. Calls are asynchronous on
 * `stream`, use no atomics (bitwise reproducible) and allocate nothing; every check happens
 * before any HIP call. Status codes are those of ssm_scan.h.
 */
#ifndef SSM_CONV_H
#define SSM_CONV_H

#include <stdint.h>

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* flags: the storage type (SSM_IO_F32 or SSM_IO_BF16), and */
#define SSM_CONV_SILU (1u << 11)

/*
 * ssm_conv_fwd -- the convolution of a prompt, described above.
 * Required: x, weight, out (each may be NULL only when its array is empty). Optional (NULL):
 * bias, initial_state, lengths, final_state (not returned).
 * batch, dim, seqlen >= 0; width 2, 3 or 4. seqlen == 0 leaves out untouched and sets
 * final_state to the initial state. out and final_state must overlap no other argument (a
 * strided array counts with its whole extent).
 * Returns SSM_OK, SSM_ERR_INVALID_ARG, SSM_ERR_UNSUPPORTED (width, a storage type other than
 * fp32/bf16, neither stride 1, batch above 65535, batch*dim or seqlen above 2^31 - 1, or more
 * than a grid of 2^32 - 1 work-items takes: a batch row of some 2^35 elements, a gradient of
 * 2^28 / (width + 1) channels), SSM_ERR_MISALIGNED (a pointer not aligned to its element size)
 * or SSM_ERR_HIP.
 */
SSM_API int ssm_conv_fwd(const void* x, const int64_t* x_strides, const float* weight,
                         const float* bias, const void* initial_state, const int32_t* lengths,
                         uint32_t flags, void* out, void* final_state, int64_t batch,
                         int64_t dim, int64_t width, int64_t seqlen, void* stream);

/*
 * ssm_conv_bwd -- gradients of L = sum(dout * out) + sum(dfinal * final_state).
 * Inputs: the forward's, dout, dfinal (NULL: zero). Outputs, overwritten: dx (0 at and behind
 * a row's length), dweight, dbias (NULL: not wanted), dinitial (NULL: not wanted; the gradient
 * of initial_state, also where that is NULL and taken as zero).
 * workspace: ssm_conv_bwd_workspace_bytes(batch, dim, width, seqlen, flags) bytes
 * (workspace_bytes, at least that), 256-byte aligned, overwritten; calls that share it must
 * not overlap in time. The sums over steps and batch rows are added in a fixed order.
 * The outputs and the workspace must overlap no other argument. Errors as ssm_conv_fwd, plus
 * SSM_ERR_INVALID_ARG for a workspace that is too small.
 */
SSM_API int ssm_conv_bwd(const void* x, const int64_t* x_strides, const float* weight,
                         const float* bias, const void* initial_state, const int32_t* lengths,
                         uint32_t flags, const void* dout, const void* dfinal, void* dx,
                         const int64_t* dx_strides, float* dweight, float* dbias,
                         void* dinitial, void* workspace, int64_t workspace_bytes,
                         int64_t batch, int64_t dim, int64_t width, int64_t seqlen,
                         void* stream);

/* Bytes of workspace ssm_conv_bwd needs (either order of x): a partial sum of every weight and
 * bias per batch row and run of steps. -1 for negative sizes, a width outside 2..4, an unknown
 * storage type or a size past int64. */
SSM_API int64_t ssm_conv_bwd_workspace_bytes(int64_t batch, int64_t dim, int64_t width,
                                             int64_t seqlen, uint32_t flags);

/*
 * ssm_conv_step -- one step of `batch` rows against a cache of past inputs.
 *   x    : [batch, dim] storage type, rows x_stride elements apart, channels contiguous
 *   state: [nslots, dim, W-1] contiguous, storage type, updated in place: row i reads the
 *          window of slot s = slots[i] (s = i if slots is NULL), then drops its oldest input
 *          and appends x[i]
 *   slots: [batch] int32, or NULL (then nslots >= batch)
 *   out  : [batch, dim] contiguous
 * A row whose slot lies outside [0, nslots) (-1, say: the padding of a captured batch) has no
 * state: its out is 0 and nothing else is written. Rows naming the same slot are successive
 * tokens of it, in row order. out and state must overlap no other argument. Errors as
 * ssm_conv_fwd.
 */
SSM_API int ssm_conv_step(const void* x, int64_t x_stride, void* state, const float* weight,
                          const float* bias, const int32_t* slots, uint32_t flags, void* out,
                          int64_t batch, int64_t nslots, int64_t dim, int64_t width,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_CONV_H */
