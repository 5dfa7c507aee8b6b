/*
 * mcc1d_delta.h - the gated delta rule, for prompts (with its gradients) and
 * for single tokens. Part of libmcc1d.so; status codes and dtypes are those of
 * mcc1d.h.
 *
 * H heads of V values keep a state S [V,K] each; H/G of them share one of G
 * heads of queries and keys. For every sequence and head, token by token:
 *
 *   a(t) = exp(A dt(t)),  dt(t) = softplus(delta(t) + delta_bias)   (MCC1D_SOFTPLUS),
 *          or delta(t) + delta_bias; 1 without delta (A and delta_bias are not read)
 *   b(t) = sigmoid(beta(t))   (MCC1D_SIGMOID), or beta(t)
 *   k'(t) = k(t) / sqrt(|k(t)|^2 + 1e-6),  q'(t) = scale q(t) / sqrt(|q(t)|^2 + 1e-6)
 *          (MCC1D_QK_NORM), or k(t) and scale q(t)
 *   u(t) = b(t) (v(t) - a(t) S(t-1) k'(t))
 *   S(t) = a(t) S(t-1) + u(t) k'(t)^T,   y(t) = S(t) q'(t)
 *   with S(-1) = `state`, or zero.
 *
 * Conventions:
 *  - 16-bit tensors (bf16 or fp16, one dtype per call): q, k, v, delta, beta, y
 *    and their gradients. fp32 tensors: A, delta_bias [H], the states [B,H,V,K]
 *    and their gradients. Sums and states are fp32, or what is as near; an
 *    output is rounded once, to nearest even.
 *  - q, k [S,B,G,K] and v, grad_y [S,B,H,V] take explicit strides in elements
 *    for S, B and the heads, their last axis adjacent; delta, beta [S,B,H] take
 *    strides for S and B, H adjacent (single tokens: without the strides for
 *    S). Strides may be zero and of any alignment, rows of 16-byte alignment
 *    move faster; negative strides are refused. Everything else, and every
 *    output, is dense.
 *  - `lengths` (int32 [B], on the device) or NULL: sequence b ends after
 *    lengths[b] tokens (values outside 0..S are taken as the nearer end).
 *    Tokens past the end are not read: their outputs and gradients are zero,
 *    and the final state is the one after the last token (the initial state
 *    for a length of zero).
 *  - `slots` (int32 [B], on the device) or NULL: row b of a single-token call
 *    updates row slots[b] of the cache `state` [cache_rows,H,V,K] in place; a
 *    value outside 0..cache_rows-1 marks a padding row, whose y is zero and
 *    which touches no state. Two rows must not name one slot. NULL means row b
 *    updates cache row b.
 *  - Pointers are DEVICE pointers owned by the caller, with the alignment of
 *    their element. Outputs must not overlap inputs or each other (a step's
 *    `state` is both). The library allocates nothing and keeps nothing between
 *    calls; what a call needs is in `workspace` (16-byte aligned), sized by the
 *    *_workspace_size call, whose contents on entry are ignored. With c chunks of 64
 *    tokens it is 35840 c B H bytes for prompts (none below 32 tokens), and 8 S B H V
 *    + c B H (8 K V + 55296) for gradients: 1.0 GB for 16 K tokens of 16 heads of 128
 *    x 128. Where B H is small, up to 63 states and K x K matrices of each are added.
 *  - Every call enqueues on `stream` of the current device and returns without
 *    waiting. Results are deterministic: no floating-point atomics, every sum
 *    in an order that depends on the shape only.
 *  - Limits: 1 <= S <= 2^31 - 4096, 1 <= B <= 65535, 1 <= H <= 2^20,
 *    H % G == 0, 1 <= K <= 128, 1 <= V <= 1024, and B*H*V*K, B*H*V and a
 *    grid's blocks below 2^31; scale is a number in fp32.
 *  - Range: a decay above one is taken, as long as 64 tokens together grow a state
 *    by less than 2^126; a token's decay counts as 2^-255 at least. Prompts of 32
 *    tokens or more go in chunks of 64 through the tensor cores, in rows of 22 bits.
 *    With growth, outputs are off by the rounding of what the decays alone would
 *    make of states and values, also where keys overwrite most of it token by token
 *    (one key, or few); b |k|^2 above 2, which turns a state over on itself, is
 *    growth too. A row of a state keeps its accuracy beside louder rows, and while
 *    it fades by up to 2^34 in a chunk. What is left of it, of a value or of grad_y
 *    after it has faded by more within one chunk, with nothing added since, is off
 *    by up to 2^-57 of what it was (a gradient of the state on its way through the
 *    chunk by its own rounding, however small it has become). Values below 2^-100
 *    are off by up to 2^-125, keys of one token by 2^-40 of the largest of them.
 *    Squares of q and k (MCC1D_QK_NORM) are summed in fp32.
 *  - Values that are not finite make NaN or infinity of the outputs that depend on
 *    them, and of no others: of a token's q of its y; of its v of one row of y and
 *    the state from that token on; of k, delta, beta, A and delta_bias of all rows of
 *    the head from there on. Gradients hide none, but may be NaN for the chunk of 64
 *    tokens where the definition's are not yet.
 *
 * Errors as in mcc1d_ssm.h.
 */
#ifndef MCC1D_DELTA_H
#define MCC1D_DELTA_H

#include <stdint.h>

#include "mcc1d.h"
#include "mcc1d_ssm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags of a call, beside MCC1D_SOFTPLUS. */
enum { MCC1D_SIGMOID = 8, MCC1D_QK_NORM = 16 };

/* Over prompts. Required: q, k, v, beta, y; A with delta. */
typedef struct mcc1d_delta_args {
    const void *q;              /* [S,B,G,K] */
    int64_t q_strides[3];       /* S, B, G */
    const void *k;              /* [S,B,G,K] */
    int64_t k_strides[3];
    const void *v;              /* [S,B,H,V] */
    int64_t v_strides[3];       /* S, B, H */
    const void *delta;          /* [S,B,H] or NULL */
    int64_t delta_strides[2];   /* S, B */
    const void *beta;           /* [S,B,H] */
    int64_t beta_strides[2];
    const float *A;             /* [H] */
    const float *delta_bias;    /* [H] or NULL */
    const float *state;         /* [B,H,V,K] or NULL */
    const int32_t *lengths;     /* [B] or NULL */
    void *y;                    /* [S,B,H,V] out */
    float *final_state;         /* [B,H,V,K] out, or NULL */
    int64_t S, B, H, G, K, V;
    double scale;
    int32_t dtype, flags;
} mcc1d_delta_args;

int32_t mcc1d_delta_workspace_size(const mcc1d_delta_args *a, uint64_t *bytes_out);
int32_t mcc1d_delta(const mcc1d_delta_args *a, void *workspace, uint64_t workspace_bytes, void *stream);

/* Its gradients, of any loss with gradient grad_y of y and grad_final_state of
 * the final state. `fwd` holds the forward's inputs (its y and final_state are
 * ignored). Required: grad_y, grad_q, grad_k, grad_v, grad_beta, and grad_delta
 * and grad_A with delta; grad_delta_bias needs delta_bias and may be NULL;
 * grad_state is optional, with or without a state. */
typedef struct mcc1d_delta_bwd_args {
    mcc1d_delta_args fwd;
    const void *grad_y;         /* [S,B,H,V] */
    int64_t grad_y_strides[3];
    const float *grad_final_state; /* [B,H,V,K] or NULL */
    void *grad_q, *grad_k;      /* [S,B,G,K] out */
    void *grad_v;               /* [S,B,H,V] out */
    void *grad_delta, *grad_beta; /* [S,B,H] out */
    float *grad_A, *grad_delta_bias; /* [H] out */
    float *grad_state;          /* [B,H,V,K] out */
} mcc1d_delta_bwd_args;

int32_t mcc1d_delta_bwd_workspace_size(const mcc1d_delta_bwd_args *a, uint64_t *bytes_out);
int32_t mcc1d_delta_bwd(const mcc1d_delta_bwd_args *a, void *workspace, uint64_t workspace_bytes, void *stream);

/* Of one token per sequence. Required: q, k, v, beta, state, y; A with delta. */
typedef struct mcc1d_delta_step_args {
    const void *q;              /* [B,G,K] */
    int64_t q_strides[2];       /* B, G */
    const void *k;              /* [B,G,K] */
    int64_t k_strides[2];
    const void *v;              /* [B,H,V] */
    int64_t v_strides[2];       /* B, H */
    const void *delta;          /* [B,H] or NULL */
    int64_t delta_stride;       /* B */
    const void *beta;           /* [B,H] */
    int64_t beta_stride;
    const float *A;             /* [H] */
    const float *delta_bias;    /* [H] or NULL */
    float *state;               /* [cache_rows,H,V,K], updated in place */
    const int32_t *slots;       /* [B] or NULL */
    void *y;                    /* [B,H,V] out */
    int64_t cache_rows, B, H, G, K, V;
    double scale;
    int32_t dtype, flags;
} mcc1d_delta_step_args;

int32_t mcc1d_delta_step(const mcc1d_delta_step_args *a, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MCC1D_DELTA_H */
