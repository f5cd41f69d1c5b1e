/*
 * ssm_linattn.h -- C ABI of linear attention with a decay for each head in libssmscan.so (gfx950):
 * a prompt in chunks, its gradient, and one token of many requests against a cache of states. It
 * is the recurrence of ssm_ssd.h (ybb.press/ai-applications/14118.html, section 2.2) with a key
 * (B) and a query (C) for each head or group of heads, any head sizes, and a gradient.
 *
 * For batch row b, head h of v (its query and key head h / (heads / qk_heads)) and step t:
 *
 *   S_t   = exp(g_t) S_{t-1} + v_t k_t^T          (g NULL: no decay)
 *   out_t = scale S_t q_t
 *
 * and behind a row's length the state stays and out is 0. In chunks of 64 steps (fp32: 32) with
 * cs_t the running sum of g, as in mhpq.cn/news/1077344 (section 5.2):
 *
 *   out_t = scale sum_{s<=t} exp(cs_t - cs_s) (q_t . k_s) v_s + scale exp(cs_t) S_in q_t
 *   S_out = exp(cs_end) S_in + sum_s exp(cs_end - cs_s) v_s k_s^T
 *
 * Memory: device pointers owned by the caller.
 *   q, k      : [batch, seqlen, qk_heads, dk]   storage type, strided
 *   v, dout   : [batch, seqlen, heads, dv]      storage type, strided
 *               *_strides: three element strides (batch, step, head) of an array whose last axis is
 *               contiguous, or NULL: the array is contiguous. The strides may be 0 or overlap.
 *   g         : [batch, seqlen, heads] fp32 with strides g_strides (NULL: contiguous); {0, 0, 1}: one
 *               log decay for each head. Values below -1e4 count as -1e4, whose decay is 0 all the
 *               same (a reset).
 *   initial_state, final_state, dfinal, dinitial : [batch, heads, dv, dk] fp32, contiguous
 *   lengths   : [batch] int32, the steps of each row (clamped to [0, seqlen]); q, k, v, g and dout
 *               behind them are not read
 *   out, dq, dk, dv : contiguous, storage type
 * Storage type (flags): SSM_IO_F32 or SSM_IO_BF16. Sums and states are fp32, sums of log decays
 * 64-bit; with bf16 storage the weights of the pairs of a chunk are rounded to bf16 once as operands
 * of the matrix cores, and the states enter as two or three bf16 pieces.
 *
 * A NaN or infinity is in the results that the recurrence and its adjoint take it to, and in no
 * other: of the forward, those of its own and later steps. Where the recurrence gives an infinity, a
 * result may be NaN: with bf16 storage an infinite v, or a state above 3.39e38, gives NaN.
 *
 * Results and workspace must overlap no other argument. Calls are asynchronous on `stream`, use
 * no atomics (bitwise reproducible) and allocate nothing; every check happens before any HIP call.
 * Calls that share a workspace must not overlap in time. Return SSM_OK, SSM_ERR_INVALID_ARG (also a
 * workspace too small, heads no multiple of qk_heads), SSM_ERR_UNSUPPORTED (dk or dv outside [1, 256],
 * batch above 65535, steps of an array 16 MiB apart or more, sizes past int64 or a grid of 2^32 - 1
 * work-items, a storage type other than fp32/bf16), SSM_ERR_MISALIGNED (a pointer not aligned to its
 * element size, a workspace not to 256 bytes) or SSM_ERR_HIP.
 */
#ifndef SSM_LINATTN_H
#define SSM_LINATTN_H

#include <stdint.h>

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The gradient's flag: dg is [heads], the sum over batch rows and steps. */
#define SSM_LINATTN_HEAD_DG (1u << 13)

/* Bytes of workspace of the forward (0 where the rows and heads fill the device) and of the
 * gradient (two fp32 states for every chunk); -1 for sizes that no call takes. */
SSM_API int64_t ssm_linattn_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads,
                                                int64_t dk, int64_t dv, uint32_t flags);
SSM_API int64_t ssm_linattn_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t heads,
                                                int64_t dk, int64_t dv, uint32_t flags);

/* Optional (NULL): g, initial_state, lengths, final_state. seqlen 0 sets final_state to the
 * initial one. */
SSM_API int ssm_linattn_fwd(const void* q, const int64_t* q_strides, const void* k,
                            const int64_t* k_strides, const void* v, const int64_t* v_strides,
                            const float* g, const int64_t* g_strides, const float* initial_state,
                            const int32_t* lengths, float scale, uint32_t flags, void* out,
                            float* final_state, void* workspace, int64_t workspace_bytes,
                            int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads,
                            int64_t dk, int64_t dv, void* stream);

/* Gradients of sum(dout * out) + sum(dfinal * final_state). Optional (NULL): g, initial_state,
 * lengths, dfinal, dg (which needs g), dinitial. dq_out and dk_out: [batch, seqlen, qk_heads, dk], the
 * sums over the heads that share a query and key; dv_out as v; dg [batch, seqlen, heads] or, with
 * SSM_LINATTN_HEAD_DG, [heads]. Behind a row's length they are 0. */
SSM_API int ssm_linattn_bwd(const void* q, const int64_t* q_strides, const void* k,
                            const int64_t* k_strides, const void* v, const int64_t* v_strides,
                            const void* dout, const int64_t* dout_strides, const float* g,
                            const int64_t* g_strides, const float* initial_state,
                            const int32_t* lengths, const float* dfinal, float scale,
                            uint32_t flags, void* dq_out, void* dk_out, void* dv_out, float* dg,
                            float* dinitial, void* workspace, int64_t workspace_bytes,
                            int64_t batch, int64_t seqlen, int64_t qk_heads, int64_t heads,
                            int64_t dk, int64_t dv, void* stream);

/*
 * One token: q, k [batch, qk_heads, dk], v [batch, heads, dv] with two strides (batch, head; NULL:
 * contiguous); g [batch, heads] with strides g_strides (NULL: contiguous; {0, 1}: one for each
 * head) or NULL; state [nslots, heads, dv, dk] fp32, contiguous, updated in place; slots [batch]
 * int32, the slot of each row, or NULL (row i is slot i; then nslots >= batch); out [batch, heads,
 * dv] contiguous. A row whose slot lies outside [0, nslots) has no state: its out is 0 and
 * nothing else is written. Rows naming the same slot are successive tokens of it, in row order.
 */
SSM_API int ssm_linattn_step(const void* q, const int64_t* q_strides, const void* k,
                             const int64_t* k_strides, const void* v, const int64_t* v_strides,
                             const float* g, const int64_t* g_strides, const int32_t* slots,
                             float scale, uint32_t flags, float* state, void* out, int64_t batch,
                             int64_t nslots, int64_t qk_heads, int64_t heads, int64_t dk,
                             int64_t dv, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_LINATTN_H */
