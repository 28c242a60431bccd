/*
 * groupnorm.h -- C ABI of the group norm, channels last, in libwkv7.so (AMD
 * MI355X, gfx950): the norm of a recurrence's heads, with the activation and
 * the output gate that follow it.
 *
 *     xh = (x - mean) * rstd,  rstd = 1 / sqrt(var + eps)     over T positions and C / G channels
 *     y  = act(xh * weight + bias) * gate                     act: none or silu
 *
 * x, gate, y [B, T, C]; group g has the channels g C / G ... ; mean and variance
 * (of the whole population) are those of each (b, g).  T = 1 normalises every
 * row by itself: a recurrence's output [batch, tokens, H, D] is [batch * tokens,
 * 1, H D] with G = H here.
 *
 * The gate is for act(norm) * gate only.  A layer that adds something between the norm and
 * the gate, such as a bonus of the token itself, calls this without a gate, adds, and gates
 * by itself; wkv7_forward's r_k adds its bonus to y, so before any norm that follows.
 *
 * weight, bias [C] fp32 (NULL: 1 and 0); gate of in_dtype or NULL; mean, rstd
 * [B, G] fp32.
 *
 * Ragged batches (desc->lengths): positions t >= lengths[b] are padding: they do
 * not count in the statistics, and their y and gradients are 0.  A sequence
 * without positions has mean 0 and rstd 1 / sqrt(eps).
 *
 * Ownership, streams, errors, overlaps: as in ssm.h.
 */
#ifndef GROUPNORM_H
#define GROUPNORM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum groupnorm_act { GROUPNORM_NONE = 0, GROUPNORM_SILU = 1 };

typedef struct groupnorm_desc {
    int32_t B;        /* batch, >= 0 */
    int32_t T;        /* positions, >= 0 */
    int32_t C;        /* channels, >= 0 */
    int32_t G;        /* groups, > 0, C % G == 0 */
    int32_t in_dtype; /* wkv7_dtype of x and gate */
    int32_t y_dtype;  /* wkv7_dtype of y (and of dy in the backward) */
    int32_t act;      /* groupnorm_act */
    float   eps;      /* > 0, finite */
    const int32_t* lengths; /* [B] device int32, 4-byte aligned, or NULL */
} groupnorm_desc;

/* Workspace bytes of groupnorm_forward: partial statistics of groups that are too large for the registers of
 * one wave (T = 1) or one workgroup (T > 1).  0 when there is nothing to compute, and at T = 1 for groups of up
 * to 1024 channels, of up to 2048 where their number is even.  Host only. */
int64_t groupnorm_workspace_bytes(const groupnorm_desc* desc);

/* y, and mean and rstd where they are not NULL (both or neither). */
int groupnorm_forward(const groupnorm_desc* desc, const void* x, const float* weight, const float* bias,
                      const void* gate, void* y, float* mean, float* rstd,
                      void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of groupnorm_backward; 0 when B T C == 0.  Host only. */
int64_t groupnorm_backward_workspace_bytes(const groupnorm_desc* desc);

/* The gradients of <dy, y>, with mean and rstd as the forward wrote them: dx [B, T, C] of
 * in_dtype; dweight, dbias [C] fp32, each may be NULL where weight or bias is; dgate of in_dtype
 * exactly when gate is given. */
int groupnorm_backward(const groupnorm_desc* desc, const void* x, const float* weight, const float* bias,
                       const void* gate, const void* dy, const float* mean, const float* rstd,
                       void* dx, float* dweight, float* dbias, void* dgate,
                       void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GROUPNORM_H */
