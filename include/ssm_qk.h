/*
 * ssm_qk.h -- C ABI of the norm of every head's queries and keys with the position rotation in the
 * same pass, in libssmscan.so (gfx950), ahead of the linear attention of ssm_linattn.h.
 *
 * For every head of every step, x of dim values, w its side's weight (NULL: ones):
 *
 *   y   = w x / sqrt(mean(x^2) + eps)
 *   out = y with the pairs (a, b) of its first rot values turned by the step's position p:
 *         (a cos - b sin, b cos + a sin), cos and sin at [p, i] for pair i
 *         pairs (i, i + rot / 2), or with SSM_QK_INTERLEAVED (2 i, 2 i + 1)
 *
 * Memory: device pointers owned by the caller.
 *   q [batch, seqlen, q_heads, dim], k [batch, seqlen, k_heads, dim] (and dq_out, dk_out, the gradients
 *               of the results): storage type; *_strides: three element strides (batch, step,
 *               head) of an array whose last axis is contiguous, or NULL: contiguous
 *   q_weight, k_weight : [dim] fp32 or NULL
 *   cos, sin  : [table_rows, rot / 2] fp32, contiguous (NULL where rot is 0)
 *   positions : [batch, seqlen] int32, or NULL: step t is at position t. A step whose position
 *               lies outside [0, table_rows) (-1, say: padding) gives zeros, and no gradient;
 *               where rot is 0 there is no table, and only positions below 0 are outside.
 *   q_out, k_out, dq, dk : contiguous, storage type;  dq_weight, dk_weight : [dim] fp32
 * Arithmetic is fp32; results are rounded once. mean(x^2) has to be finite in fp32.
 *
 * Results and workspace must overlap no other argument. Calls are asynchronous on `stream`,
 * bitwise reproducible, and allocate nothing; every check happens before any HIP call. Return SSM_OK,
 * SSM_ERR_INVALID_ARG (also a workspace too small), SSM_ERR_UNSUPPORTED (dim outside [1, 256], rot odd
 * or outside [0, dim], sizes past int64 or a grid of 2^32 - 1 work-items, a storage type other than
 * fp32/bf16), SSM_ERR_MISALIGNED (a pointer not aligned to its element size, a workspace not to
 * 256 bytes) or SSM_ERR_HIP.
 */
#ifndef SSM_QK_H
#define SSM_QK_H

#include <stdint.h>

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_QK_INTERLEAVED (1u << 14)

SSM_API int ssm_qk_norm_fwd(const void* q, const int64_t* q_strides, const void* k,
                            const int64_t* k_strides, const float* q_weight,
                            const float* k_weight, const float* cos, const float* sin,
                            const int32_t* positions, float eps, uint32_t flags, void* q_out,
                            void* k_out, int64_t batch, int64_t seqlen, int64_t q_heads,
                            int64_t k_heads, int64_t dim, int64_t rot, int64_t table_rows,
                            void* stream);

/* Bytes of workspace of the gradient; -1 for sizes that no call takes. */
SSM_API int64_t ssm_qk_norm_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t q_heads,
                                                int64_t k_heads, int64_t dim, int64_t rot,
                                                uint32_t flags);

/* Gradients of sum(dq_out * q_out) + sum(dk_out * k_out). dq_weight and dk_weight may be NULL. */
SSM_API int ssm_qk_norm_bwd(const void* q, const int64_t* q_strides, const void* k,
                            const int64_t* k_strides, const void* dq_out,
                            const int64_t* dq_out_strides, const void* dk_out,
                            const int64_t* dk_out_strides, const float* q_weight,
                            const float* k_weight, const float* cos, const float* sin,
                            const int32_t* positions, float eps, uint32_t flags, void* dq,
                            void* dk, float* dq_weight, float* dk_weight, void* workspace,
                            int64_t workspace_bytes, int64_t batch, int64_t seqlen,
                            int64_t q_heads, int64_t k_heads, int64_t dim, int64_t rot,
                            int64_t table_rows, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_QK_H */
