/*
 * ssm.h -- C ABI of the selective state space scan in libwkv7.so (AMD MI355X,
 * gfx950): a recurrence with a diagonal state whose step size, input and
 * readout vectors come with every token.
 *
 * Per batch b and channel c, with N states, over tokens t:
 *
 *     d_t = softplus(dt_t + dt_bias)                         (or dt_t + dt_bias)
 *     h_t = exp(d_t A) h_{t-1} + d_t x_t Bm_t                (state n: A[c][n], Bm_t[g][n])
 *     y_t = (sum_n Cm_t[g][n] h_t[n] + D x_t) * silu(z_t)    (D, z optional)
 *
 * Channels come in G groups of C / G consecutive ones; a group shares Bm and Cm.
 * Runs of 16 tokens are composed from what they do to any incoming state, so a
 * growing state (d_t A > 0) has to grow by a finite fp32 factor over 16 tokens.
 *
 * Layouts (row-major, contiguous):
 *     x, dt, z, y : [B, T, C]            Bm, Cm : [B, T, G, N]
 *     A           : [C, N] fp32 (the rates themselves, negative for a decaying state)
 *     D, dt_bias  : [C] fp32, each NULL for zero
 *     states      : [B, C, N] fp32
 * x, dt, z, Bm, Cm have desc->in_dtype; states, sums and parameters are fp32.
 *
 * Ragged batches (desc->lengths): tokens t >= lengths[b] of sequence b are
 * padding: they leave the state as it was, their y is 0, and their gradients
 * are 0; nothing about their input values matters.  A length below 0 counts as
 * 0, one above T as T.
 *
 * Ownership, streams, errors: as in wkv7.h (caller-owned, 16-byte aligned
 * device pointers; work enqueued on `stream`; WKV7_* status codes with
 * wkv7_last_error() for details; all checks before any HIP call; nothing is
 * allocated or kept).  Every array that a call writes shares no byte with any
 * other array of that call (EINVAL), except where in place is allowed.
 * Results do not depend on the order in which the device runs the workgroups.
 */
#ifndef SSM_H
#define SSM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ssm_desc {
    int32_t B;           /* batch, >= 0 */
    int32_t T;           /* tokens, >= 0 (ssm_step: 1) */
    int32_t C;           /* channels, >= 0 */
    int32_t N;           /* states per channel, 1 .. 64 (larger: EUNSUPPORTED) */
    int32_t G;           /* channel groups, C % G == 0 (0 means 1) */
    int32_t in_dtype;    /* wkv7_dtype of x, dt, z, Bm, Cm */
    int32_t y_dtype;     /* wkv7_dtype of y (and of dy in the backward) */
    int32_t dt_softplus; /* 1: d = softplus(dt + dt_bias); 0: d = dt + dt_bias */
    int32_t S;           /* ssm_step: states in the pool; ignored elsewhere */
    int32_t reserved;    /* 0 */
    const int32_t* lengths; /* [B] device int32, 4-byte aligned, or NULL: every sequence has T tokens
                               (ssm_step: must be NULL) */
} ssm_desc;

/* Tokens from one checkpointed state to the next. */
#define SSM_CHECKPOINT_TOKENS 32

/* Bytes of the states that ssm_forward can leave for ssm_backward: [B][ceil(T / 32)][C][N]
 * fp32, the state before every 32nd token.  A negative wkv7_status if the
 * descriptor is invalid.  Host only. */
int64_t ssm_checkpoint_bytes(const ssm_desc* desc);

/* y over T tokens from state_in (or zeros); state_out (may be NULL) gets the state after
 * the last token of each sequence.  state_in == state_out is allowed.  T == 0 copies
 * state_in (or zeros) to state_out.  checkpoints: NULL, or ssm_checkpoint_bytes(desc)
 * bytes that the call fills for ssm_backward. */
int ssm_forward(const ssm_desc* desc, const void* x, const void* dt, const float* A,
                const void* Bm, const void* Cm, const float* D, const float* dt_bias,
                const void* z, const float* state_in, void* y, float* state_out,
                float* checkpoints, void* stream);

/* One token per row, on a pool of states: x, dt, z, y [B, C], Bm, Cm [B, G, N], state
 * [S, C, N] updated in place.  Row b works on state state_index[b] (NULL: on state b;
 * then S >= B).  A row whose index is outside 0 .. S - 1 has no request: its y is 0 and no
 * state is touched.  Where an index comes twice, the first of the rows has it and the later
 * ones are treated as rows without a request. */
int ssm_step(const ssm_desc* desc, const void* x, const void* dt, const float* A,
             const void* Bm, const void* Cm, const float* D, const float* dt_bias,
             const void* z, float* state, const int32_t* state_index, void* y, void* stream);

/* Workspace bytes of ssm_backward for this descriptor; without_checkpoints != 0: for a call
 * that has none (it then runs the forward's recurrence first, into the workspace).  0 when
 * B T C == 0.  A negative wkv7_status if the descriptor is invalid.  Host only. */
int64_t ssm_backward_workspace_bytes(const ssm_desc* desc, int without_checkpoints);

/* The gradients of <dy, y> + <dstate_out, state_out> for ssm_forward with these inputs.
 *   dy          : [B, T, C] of y_dtype
 *   dstate_out  : [B, C, N] fp32 or NULL (zero)
 *   checkpoints : as ssm_forward filled them for the same inputs and state_in, or NULL
 *   dx, ddt, dz : [B, T, C] of in_dtype (dz exactly when z is given)
 *   dBm, dCm    : [B, T, G, N] of in_dtype, summed over a group's channels
 *   dA          : [C, N] fp32, dD, ddt_bias : [C] fp32, summed over the batch; dD and
 *                 ddt_bias may be NULL (not computed) and have to be where D or dt_bias is
 *   dstate_in   : [B, C, N] fp32 or NULL (not computed)
 *   workspace   : at least ssm_backward_workspace_bytes(desc, checkpoints == NULL) bytes.
 * T == 0: the parameters' gradients are 0 and dstate_in is dstate_out (or 0). */
int ssm_backward(const ssm_desc* desc, const void* x, const void* dt, const float* A,
                 const void* Bm, const void* Cm, const float* D, const float* dt_bias,
                 const void* z, const float* state_in, const void* dy, const float* dstate_out,
                 const float* checkpoints, void* dx, void* ddt, float* dA, void* dBm, void* dCm,
                 float* dD, float* ddt_bias, void* dz, float* dstate_in,
                 void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_H */
