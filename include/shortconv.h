/*
 * shortconv.h -- C ABI of the short causal convolution in libwkv7.so (AMD
 * MI355X, gfx950): every channel is filtered by its own K taps over the tokens,
 * as in front of a recurrence.
 *
 *     y_t = act(bias + sum_{k < K} w[c][k] x_{t - K + 1 + k}),    act: none or silu
 *
 * The inputs before the first token come from a state: the last K - 1 inputs
 * that the sequence has had, oldest first (NULL: zeros).
 *
 * Layouts (row-major, contiguous): x, y [B, T, C]; w [C, K] fp32; bias [C] fp32
 * or NULL; states [B, K - 1, C] of in_dtype (they hold inputs, unrounded);
 * their gradients [B, K - 1, C] fp32.
 *
 * Ragged batches (desc->lengths) as in ssm.h: tokens t >= lengths[b] are
 * padding, y and gradients 0 there, and state_out holds the last K - 1 inputs of
 * the sequence itself (reaching into state_in where it is shorter).
 *
 * Ownership, streams, errors, overlaps: as in ssm.h.
 */
#ifndef SHORTCONV_H
#define SHORTCONV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum shortconv_act { SHORTCONV_NONE = 0, SHORTCONV_SILU = 1 };

typedef struct shortconv_desc {
    int32_t B;        /* batch, >= 0 */
    int32_t T;        /* tokens, >= 0 (shortconv_step: 1) */
    int32_t C;        /* channels, >= 0 */
    int32_t K;        /* taps: 2, 3 or 4 (others EUNSUPPORTED) */
    int32_t in_dtype; /* wkv7_dtype of x and the states */
    int32_t y_dtype;  /* wkv7_dtype of y (and of dy in the backward) */
    int32_t act;      /* shortconv_act */
    int32_t S;        /* shortconv_step: states in the pool; ignored elsewhere */
    const int32_t* lengths; /* [B] device int32, 4-byte aligned, or NULL (shortconv_step: must be NULL) */
} shortconv_desc;

/* y over T tokens; state_out (may be NULL) gets the last K - 1 inputs.
 * state_in == state_out is allowed.  T == 0 copies state_in (or zeros) to state_out. */
int shortconv_forward(const shortconv_desc* desc, const void* x, const float* w, const float* bias,
                      const void* state_in, void* y, void* state_out, void* stream);

/* One token per row on a pool of states, state [S, K - 1, C] updated in place;
 * state_index as in ssm_step. */
int shortconv_step(const shortconv_desc* desc, const void* x, const float* w, const float* bias,
                   void* state, const int32_t* state_index, void* y, void* stream);

/* Workspace bytes of shortconv_backward; 0 when B T C == 0.  Host only. */
int64_t shortconv_backward_workspace_bytes(const shortconv_desc* desc);

/* The gradients of <dy, y> + <dstate_out, state_out>: dx [B, T, C] of in_dtype,
 * dw [C, K] fp32, dbias [C] fp32 or NULL (required with bias), dstate_in
 * [B, K - 1, C] fp32 or NULL.  T == 0: dw and dbias are 0 and dstate_in is dstate_out (or 0). */
int shortconv_backward(const shortconv_desc* desc, const void* x, const float* w, const float* bias,
                       const void* state_in, const void* dy, const float* dstate_out,
                       void* dx, float* dw, float* dbias, float* dstate_in,
                       void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SHORTCONV_H */
