/*
 * linattn.h -- C ABI of linear attention with a decay for each head in libwkv7.so
 * (AMD MI355X, gfx950): a matrix state per head that decays by one factor a token
 * and takes up the token's key and value.
 *
 * Per batch b and head h, with S of Dk x Dv, over tokens t:
 *
 *     S_t = exp(g_t) S_{t-1} + k_t v_t^T
 *     y_t = scale S_t^T q_t
 *
 * Heads: H for g, y and the states; q has Hq, k has Hk and v has Hv heads, each a divisor
 * of H: head h uses head h / (H / Hq) of q, and so on.
 *
 * Layouts (row-major, contiguous):
 *     q [B, T, Hq, Dk]   k [B, T, Hk, Dk]   v [B, T, Hv, Dv]   y [B, T, H, Dv]
 *     g : the logarithm of the decay, fp32, [B, T, H], or [H] (desc->g_per_token 0)
 *     states : [B, H, Dk, Dv] fp32
 * q, k and v have desc->in_dtype.
 *
 * Chunks of 64 tokens (32 where an array is fp32) are computed together, so a token that
 * is not finite, and products past fp32's range, reach every output of their chunk and the
 * ones behind it (the gradients of k and v: and the ones before it; that of g: of their 512
 * tokens and the ones before).  A growing state (g > 0) has to grow by a finite factor over a
 * chunk.  g = -inf empties a state of finite values; a g below about -1386 counts as -inf.
 *
 * Products and sums are fp32's for every type (a state is fp32, y and the gradients of q, k and
 * v are rounded once, to their type).  The gradient of g is a difference of two numbers of a
 * token, <q, dq> and <k, dk>, added up over up to 512 tokens, and is off by about 2^-19 of their
 * size whatever the difference comes to: by 1e-6 of itself where the state is kept for long,
 * 1e-5 where a token leaves exp(-2) of it, 2e-4 at exp(-5) and 4e-2 at exp(-10); further down it
 * has no right digits (its size is then below 2^-19 of the products').
 *
 * Heads of which Dk or Dv is no multiple of 8 (bf16 arrays only) or 4 are read one element at a
 * time, and take two to three times as long (a fifth to a half more where an array is fp32).
 *
 * Ragged batches (desc->lengths): tokens t >= lengths[b] of sequence b are padding: they
 * leave the state as it was, their y is 0, and their gradients are 0; nothing about their
 * input values matters.  A length below 0 counts as 0, one above T as T.
 *
 * Ownership, streams, errors, overlaps: as in ssm.h.
 */
#ifndef LINATTN_H
#define LINATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct linattn_desc {
    int32_t B;           /* batch, >= 0 */
    int32_t T;           /* tokens, >= 0 (linattn_step: 1) */
    int32_t H;           /* heads, 0 .. 16384 (more: EUNSUPPORTED) */
    int32_t Hq, Hk, Hv;  /* heads of q, k and v, divisors of H (0 means H) */
    int32_t Dk, Dv;      /* 1 .. 128 (larger: EUNSUPPORTED) */
    int32_t in_dtype;    /* wkv7_dtype of q, k, v */
    int32_t y_dtype;     /* wkv7_dtype of y (and of dy in the backward) */
    int32_t g_per_token; /* 1: g is [B, T, H]; 0: [H] */
    int32_t S;           /* linattn_step: states in the pool; ignored elsewhere */
    float   scale;       /* finite */
    int32_t reserved;    /* 0 */
    const int32_t* lengths; /* [B] device int32, 4-byte aligned, or NULL: every sequence has T tokens
                               (linattn_step: must be NULL) */
} linattn_desc;

/* Workspace bytes of linattn_forward: states between the parts of sequences that are
 * computed side by side when there are few heads; often 0.  A negative wkv7_status if the
 * descriptor is invalid.  Host only. */
int64_t linattn_workspace_bytes(const linattn_desc* desc);

/* y over T tokens from state_in (or zeros); state_out (may be NULL) gets the state after
 * the last token of each sequence.  state_in == state_out is allowed.  T == 0 copies
 * state_in (or zeros) to state_out. */
int linattn_forward(const linattn_desc* desc, const void* q, const void* k, const void* v, const float* g,
                    const float* state_in, void* y, float* state_out,
                    void* workspace, int64_t workspace_bytes, void* stream);

/* One token per row, on a pool of states: q [B, Hq, Dk], k [B, Hk, Dk], v [B, Hv, Dv],
 * g [B, H] or [H], y [B, H, Dv], state [S, H, Dk, Dv] updated in place.  state_index as in
 * ssm_step: rows without a request and later rows of the same state have y 0 and touch no
 * state. */
int linattn_step(const linattn_desc* desc, const void* q, const void* k, const void* v, const float* g,
                 float* state, const int32_t* state_index, void* y, void* stream);

/* Workspace bytes of linattn_backward; 0 when B T H is 0, and then none is touched.  Among them, for every further
 * 512 tokens behind the first, two states of each sequence and head (at widths of 64 or 128; whether or not dg is asked
 * for), and a head's gradients in fp32 where heads share q, k or v.  Host only. */
int64_t linattn_backward_workspace_bytes(const linattn_desc* desc);

/* The gradients of <dy, y> + <dstate_out, state_out> for linattn_forward with these inputs.
 *   dy         : [B, T, H, Dv] of y_dtype
 *   dstate_out : [B, H, Dk, Dv] fp32 or NULL (zero)
 *   dq, dk, dv : as q, k, v, of in_dtype, summed over the heads that share one
 *   dg         : as g, fp32, or NULL (not computed); [H]: summed over batch and tokens
 *   dstate_in  : [B, H, Dk, Dv] fp32 or NULL (not computed)
 *   workspace  : at least linattn_backward_workspace_bytes(desc) bytes.
 * dg is 0 where g counts as -inf.  T == 0: dg [H] is 0 and dstate_in is dstate_out (or 0). */
int linattn_backward(const linattn_desc* desc, const void* q, const void* k, const void* v, const float* g,
                     const float* state_in, const void* dy, const float* dstate_out,
                     void* dq, void* dk, void* dv, float* dg, float* dstate_in,
                     void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LINATTN_H */
