/*
 * layernorm.h -- C ABI of the layer norm in libwkv7.so (AMD MI355X, gfx950), with the
 * residual stream's sum in front of it: what stands before a recurrence's projections.
 *
 *     h = x + residual                                  in the stream's type (without a residual: h = x)
 *     y = (h - mean) * rstd * weight + bias,  rstd = 1 / sqrt(var + eps)     per row of C channels
 *
 * x, residual, h, y [B, T, C]; the statistics are those of h as it is stored, over a row's
 * channels (whole population).  weight, bias [C] fp32 (NULL: 1 and 0); mean, rstd [B, T] fp32.
 *
 * Types: x has x_dtype, residual and h (and their gradients) have h_dtype, y and dy have
 * y_dtype.  Without a residual h is x and h_dtype has to be x_dtype.
 *
 * Ragged batches (desc->lengths): positions t >= lengths[b] are padding: their y, h and
 * gradients are 0, and nothing about their input values matters.  Their mean is 0 and their rstd
 * 1 / sqrt(eps).
 *
 * Ownership, streams, errors, overlaps: as in ssm.h.
 */
#ifndef LAYERNORM_H
#define LAYERNORM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct layernorm_desc {
    int32_t B;        /* batch, >= 0 */
    int32_t T;        /* positions, >= 0 */
    int32_t C;        /* channels, >= 0 */
    int32_t x_dtype;  /* wkv7_dtype of x (and dx) */
    int32_t h_dtype;  /* wkv7_dtype of residual and h (and dh, dresidual) */
    int32_t y_dtype;  /* wkv7_dtype of y (and dy) */
    float   eps;      /* > 0, finite */
    int32_t reserved; /* 0 */
    const int32_t* lengths; /* [B] device int32, 4-byte aligned, or NULL */
} layernorm_desc;

/* y, and h where residual is given (h == residual, in place, is allowed; without a residual h is
 * NULL), and mean and rstd where they are not NULL (both or neither). */
int layernorm_forward(const layernorm_desc* desc, const void* x, const void* residual, const float* weight, const float* bias,
                      void* h, void* y, float* mean, float* rstd, void* stream);

/* Workspace bytes of layernorm_backward; 0 when B T C == 0.  Host only. */
int64_t layernorm_backward_workspace_bytes(const layernorm_desc* desc);

/* The gradients of <dy, y> + <dh, h>, with h, mean and rstd as the forward left them.
 *   dh        : [B, T, C] of h_dtype, what the stream's later users give, or NULL (zero)
 *   dresidual : [B, T, C] of h_dtype, the gradient of h and so of residual; dresidual == dh, in
 *               place, is allowed
 *   dx        : the same of x_dtype, or NULL (not written: where x_dtype is h_dtype, dresidual is it)
 *   dweight, dbias : [C] fp32, each may be NULL where weight or bias is
 *   workspace : at least layernorm_backward_workspace_bytes(desc) bytes. */
int layernorm_backward(const layernorm_desc* desc, const void* h, const float* weight, const float* bias,
                       const void* dy, const void* dh, const float* mean, const float* rstd,
                       void* dresidual, void* dx, float* dweight, float* dbias,
                       void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LAYERNORM_H */
