/*
 * ssm_step.h -- C ABI of the single-token state update in libssmscan.so (gfx950): one step of
 * the recurrences of ssm_scan.h (Mamba-1) and ssm_ssd.h (Mamba-2) for a batch of requests,
 * each with its state in a slot of one cache (ybb.press/ai-applications/14118.html, section
 * 5.1: a fixed-size state per layer takes the place of a growing cache).
 *
 * For row i with slot s = slots[i] (s = i if slots is NULL), channel d and state n:
 *
 *   dt        = delta[i,d] + delta_bias[d]         (Mamba-2: dt[i,h] + dt_bias[h], d's head h)
 *   dt        = softplus(dt)                       (if SSM_DELTA_SOFTPLUS)
 *   state[s,d,n] = exp(dt * A) * state[s,d,n] + dt * B[i,n] * u[i,d]
 *                                                  (A[d,n]; Mamba-2: A[h])
 *   y         = sum_n C[i,n] * state[s,d,n] + D[d] * u[i,d]        (D optional)
 *   out[i,d]  = y * z * sigmoid(z), z = z[i,d]                     (gate optional)
 *
 * Memory: device pointers owned by the caller.
 *   u (x), z   : [batch, dim]      storage type; delta: [batch, dim] (Mamba-2 dt: [batch, heads])
 *   B, C       : [batch, dstate]   storage type
 *                each with rows *_stride elements apart and its last axis contiguous
 *   A          : [dim, dstate]     fp32 (Mamba-2: [heads])
 *   D          : [dim] fp32;  delta_bias [dim], dt_bias [heads] fp32
 *   state      : [nslots, dim, dstate] fp32, contiguous, updated in place
 *   slots      : [batch] int32, or NULL (then nslots >= batch)
 *   out        : [batch, dim] contiguous, storage type
 * A row whose slot lies outside [0, nslots) (-1, say: the padding of a captured batch) has no
 * state: its out is 0 and nothing else is written. Rows naming the same slot are successive
 * tokens of it, in row order. Arithmetic is fp32; out is rounded once.
 *
 * out and state must overlap no other argument. Calls are asynchronous on `stream`, bitwise
 * reproducible, and allocate nothing; every check happens before any HIP call. Returns SSM_OK,
 * SSM_ERR_INVALID_ARG, SSM_ERR_UNSUPPORTED (dstate outside [1, 256], batch above 65535, dim or
 * nslots above 2^31 - 1, more channels than a grid of 2^32 - 1 work-items takes (2^29 of more
 * than 128 states), a storage type other than fp32/bf16, sizes past int64), SSM_ERR_MISALIGNED
 * (a pointer not aligned to its element size) or SSM_ERR_HIP.
 */
#ifndef SSM_STEP_H
#define SSM_STEP_H

#include <stdint.h>

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Mamba-1: A per channel and state, a step size per channel. */
SSM_API int ssm_scan_step(const void* u, int64_t u_stride, const void* delta,
                          int64_t delta_stride, const float* A, const void* B, int64_t b_stride,
                          const void* C, int64_t c_stride, const float* D, const void* z,
                          int64_t z_stride, const float* delta_bias, const int32_t* slots,
                          uint32_t flags, float* state, void* out, int64_t batch,
                          int64_t nslots, int64_t dim, int64_t dstate, void* stream);

/* Mamba-2: A and a step size per head of headdim channels (any headdim >= 1). */
SSM_API int ssm_ssd_step(const void* x, int64_t x_stride, const void* dt, int64_t dt_stride,
                         const float* A, const void* B, int64_t b_stride, const void* C,
                         int64_t c_stride, const float* D, const void* z, int64_t z_stride,
                         const float* dt_bias, const int32_t* slots, uint32_t flags,
                         float* state, void* out, int64_t batch, int64_t nslots,
                         int64_t nheads, int64_t headdim, int64_t dstate, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_STEP_H */
