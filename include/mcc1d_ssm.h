/*
 * mcc1d_ssm.h - the short convolution and the selective scan of a selective
 * state space layer, for prompts (with their gradients) and for single tokens.
 * Part of libmcc1d.so; status codes and dtypes are those of mcc1d.h.
 *
 * With x, u, delta, z, y laid out [S,B,H] (H adjacent), for every sequence b
 * and channel h:
 *
 *   short convolution (W taps, 1 <= W <= 8):
 *     pre(t) = bias + sum over k = 0..W-1 of weight(k) * x(t-W+1+k)
 *     y(t)   = pre(t) * sigmoid(pre(t))   (MCC1D_SILU), or pre(t)
 *     where x(t) for t = -(W-1)..-1 is the carried window (row t+W-1 of
 *     `state`), or zero without one; the final window is the last W-1 rows of
 *     the window and the sequence together.
 *
 *   selective scan (N states per channel, 1 <= N <= 64):
 *     dt(t)   = softplus(delta(t) + delta_bias)   (MCC1D_SOFTPLUS), or
 *               delta(t) + delta_bias
 *     h(t)[n] = exp(dt(t) A[n]) h(t-1)[n] + dt(t) u(t) B(t)[n]
 *     y(t)    = (sum over n of C(t)[n] h(t)[n] + D u(t)) * z(t) sigmoid(z(t))
 *     with h(-1) = `state`, or zero; without z there is no gate, without D no
 *     D term. H is cut into G equal groups of channels, each with its own
 *     B, C [S,B,G,N].
 *
 * Conventions:
 *  - 16-bit tensors (bf16 or fp16, one dtype per call): x, weight, bias, y,
 *    the convolution's windows, u, delta, z, B, C and their gradients.
 *    fp32 tensors: A [H,N], D [H], delta_bias [H], the scan's states
 *    [B,H,N] and their gradients. All arithmetic is fp32; an output is
 *    rounded once, to nearest even.
 *  - Activations [S,B,H] (single tokens: [B,H]) take explicit strides, in
 *    elements, outermost first, H always adjacent; B and C take strides for
 *    S, B and G, N adjacent. Strides may be zero and of any alignment; an
 *    input is read in place. Everything else, and every output, is dense.
 *    Negative strides are refused, as are strides of 2^31 elements and more in
 *    mcc1d_scan_step.
 *  - `lengths` (int32 [B], on the device) or NULL: sequence b ends after
 *    lengths[b] tokens (values outside 0..S are taken as the nearer end).
 *    Tokens past the end are not read: their outputs and gradients are zero,
 *    and the final state is the one after the last token (the initial state
 *    for a length of zero).
 *  - `slots` (int32 [B], on the device) or NULL: row b of a single-token call
 *    updates row slots[b] of the cache `state` [cache_rows,...] in place; a
 *    value outside 0..cache_rows-1 marks a padding row, whose y is zero and
 *    which touches no state. Two rows must not name one slot. NULL means row b
 *    updates cache row b.
 *  - Pointers are DEVICE pointers owned by the caller. Tensors may have the
 *    alignment of their element; aligned rows move faster. Outputs must not
 *    overlap inputs or each other (a step's `state` is both). The library
 *    allocates nothing and keeps nothing between calls; what a call needs is
 *    in `workspace` (256-byte aligned is best, 16 required), sized by the
 *    *_workspace_size call, whose contents on entry are ignored.
 *  - Every call enqueues on `stream` of the current device and returns
 *    without waiting. Results are deterministic: no floating-point atomics,
 *    every sum in an order that depends on the shape only.
 *  - Limits: 1 <= S <= 2^31 - 4096, 1 <= B <= 65535, 1 <= H <= 2^20,
 *    H % G == 0, and B*H*N and a grid's blocks below 2^31 (the backward's
 *    sums: S*B*G times N, padded to 4 times a power of two, below 2^37).
 *
 * Errors (nothing is enqueued): MCC1D_ERR_PARAM_NULLPTR for a null descriptor
 * or a required null pointer; MCC1D_ERR_PARAM_INVALID for a dtype, flag,
 * negative stride, an element-misaligned pointer, or an output (or the
 * workspace) that overlaps an input or another output;
 * MCC1D_ERR_INNER_TILING_ERROR for a shape outside the limits;
 * MCC1D_ERR_WORKSPACE for a workspace below the reported size;
 * MCC1D_ERR_DEVICE as in mcc1d.h; MCC1D_ERR_CUDA if a launch failed.
 */
#ifndef MCC1D_SSM_H
#define MCC1D_SSM_H

#include <stdint.h>

#include "mcc1d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flags of a call. */
enum { MCC1D_SILU = 1, MCC1D_SOFTPLUS = 2 };

/* Short convolution over prompts. Required: x, weight, y. */
typedef struct mcc1d_short_conv_args {
    const void *x;              /* [S,B,H] */
    int64_t x_strides[2];       /* S, B */
    const void *weight;         /* [W,H] */
    const void *bias;           /* [H] or NULL */
    const void *state;          /* [B,W-1,H] or NULL */
    const int32_t *lengths;     /* [B] or NULL */
    void *y;                    /* [S,B,H] out */
    void *final_state;          /* [B,W-1,H] out, or NULL */
    int64_t S, B, H, W;
    int32_t dtype, flags;
} mcc1d_short_conv_args;

int32_t mcc1d_short_conv(const mcc1d_short_conv_args *a, void *stream);

/* Its gradients, of any loss with gradient grad_y of y and grad_final_state
 * of the final window. Required: grad_y, x, weight, grad_x, grad_weight.
 * grad_bias needs bias, grad_state needs state. */
typedef struct mcc1d_short_conv_bwd_args {
    const void *grad_y;         /* [S,B,H] */
    int64_t grad_y_strides[2];
    const void *x;              /* [S,B,H] */
    int64_t x_strides[2];
    const void *weight;         /* [W,H] */
    const void *bias;           /* [H] or NULL */
    const void *state;          /* [B,W-1,H] or NULL */
    const int32_t *lengths;     /* [B] or NULL */
    const void *grad_final_state; /* [B,W-1,H] or NULL */
    void *grad_x;               /* [S,B,H] out */
    void *grad_weight;          /* [W,H] out */
    void *grad_bias;            /* [H] out, or NULL */
    void *grad_state;           /* [B,W-1,H] out, or NULL */
    int64_t S, B, H, W;
    int32_t dtype, flags;
} mcc1d_short_conv_bwd_args;

int32_t mcc1d_short_conv_bwd_workspace_size(const mcc1d_short_conv_bwd_args *a, uint64_t *bytes_out);
int32_t mcc1d_short_conv_bwd(const mcc1d_short_conv_bwd_args *a, void *workspace,
                             uint64_t workspace_bytes, void *stream);

/* Short convolution of one token per sequence. Required: x, weight, y, and
 * state for W > 1. */
typedef struct mcc1d_short_conv_step_args {
    const void *x;              /* [B,H] */
    int64_t x_stride;           /* B */
    void *state;                /* [cache_rows,W-1,H], updated in place */
    const void *weight;         /* [W,H] */
    const void *bias;           /* [H] or NULL */
    const int32_t *slots;       /* [B] or NULL */
    void *y;                    /* [B,H] out */
    int64_t cache_rows, B, H, W;
    int32_t dtype, flags;
} mcc1d_short_conv_step_args;

int32_t mcc1d_short_conv_step(const mcc1d_short_conv_step_args *a, void *stream);

/* Selective scan over prompts. Required: u, delta, A, B, C, y. */
typedef struct mcc1d_scan_args {
    const void *u;              /* [S,B,H] */
    int64_t u_strides[2];       /* S, B */
    const void *delta;          /* [S,B,H] */
    int64_t delta_strides[2];
    const void *z;              /* [S,B,H] or NULL */
    int64_t z_strides[2];
    const void *B_;             /* [S,B,G,N] */
    int64_t B_strides[3];       /* S, B, G */
    const void *C;              /* [S,B,G,N] */
    int64_t C_strides[3];
    const float *A;             /* [H,N] */
    const float *D;             /* [H] or NULL */
    const float *delta_bias;    /* [H] or NULL */
    const float *state;         /* [B,H,N] or NULL */
    const int32_t *lengths;     /* [B] or NULL */
    void *y;                    /* [S,B,H] out */
    float *final_state;         /* [B,H,N] out, or NULL */
    int64_t S, B, H, N, G;
    int32_t dtype, flags;
} mcc1d_scan_args;

int32_t mcc1d_scan_workspace_size(const mcc1d_scan_args *a, uint64_t *bytes_out);
int32_t mcc1d_scan(const mcc1d_scan_args *a, void *workspace, uint64_t workspace_bytes, void *stream);

/* Its gradients, of any loss with gradient grad_y of y and grad_final_state of
 * the final state. `fwd` holds the forward's inputs (its y and final_state are
 * ignored). Required: grad_y, grad_u, grad_delta, grad_A, grad_B, grad_C;
 * grad_z with z, grad_D with D, grad_delta_bias with delta_bias (each may also
 * be NULL); grad_state is optional, with or without a state. */
typedef struct mcc1d_scan_bwd_args {
    mcc1d_scan_args fwd;
    const void *grad_y;         /* [S,B,H] */
    int64_t grad_y_strides[2];
    const float *grad_final_state; /* [B,H,N] or NULL */
    void *grad_u, *grad_delta, *grad_z;   /* [S,B,H] out */
    void *grad_B, *grad_C;      /* [S,B,G,N] out */
    float *grad_A;              /* [H,N] out */
    float *grad_D, *grad_delta_bias;      /* [H] out */
    float *grad_state;          /* [B,H,N] out */
} mcc1d_scan_bwd_args;

int32_t mcc1d_scan_bwd_workspace_size(const mcc1d_scan_bwd_args *a, uint64_t *bytes_out);
int32_t mcc1d_scan_bwd(const mcc1d_scan_bwd_args *a, void *workspace, uint64_t workspace_bytes,
                       void *stream);

/* Selective scan of one token per sequence. Required: u, delta, A, B, C,
 * state, y. */
typedef struct mcc1d_scan_step_args {
    const void *u;              /* [B,H] */
    int64_t u_stride;           /* B */
    const void *delta;          /* [B,H] */
    int64_t delta_stride;
    const void *z;              /* [B,H] or NULL */
    int64_t z_stride;
    const void *B_;             /* [B,G,N] */
    int64_t B_strides[2];       /* B, G */
    const void *C;              /* [B,G,N] */
    int64_t C_strides[2];
    const float *A;             /* [H,N] */
    const float *D;             /* [H] or NULL */
    const float *delta_bias;    /* [H] or NULL */
    float *state;               /* [cache_rows,H,N], updated in place */
    const int32_t *slots;       /* [B] or NULL */
    void *y;                    /* [B,H] out */
    int64_t cache_rows, B, H, N, G;
    int32_t dtype, flags;
} mcc1d_scan_step_args;

int32_t mcc1d_scan_step(const mcc1d_scan_step_args *a, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MCC1D_SSM_H */
