/*
 * mcc1d_norm.h - the norms of a block of a sequence model: the one behind its
 * mixer, fused with the output gate, and the one behind the residual sum in
 * front of the next block, fused with the branch's own norm and scale. Part of
 * libmcc1d.so; status codes and dtypes are those of mcc1d.h.
 *
 *   gated norm, over the D values of each of H heads of x [S,B,H,D]:
 *     n = x / sqrt(mean(x^2) + eps),   y = n * weight * z sigmoid(z)
 *     (without z there is no gate)
 *
 *   residual norm, over the H channels of each row of x [S,B,H]:
 *     m = x / sqrt(mean(x^2) + eps) * post_weight, or x without post_weight
 *     h = residual + scale * m   (scale 1 without one)
 *     y = h / sqrt(mean(h^2) + eps) * weight     (of h before it is rounded)
 *
 * Conventions:
 *  - 16-bit tensors (bf16 or fp16, one dtype per call): x, z, y, the weights
 *    and their gradients, grad_y. residual, h and their gradients have that
 *    dtype too, or are fp32 with the flag MCC1D_WIDE. scale [H] and its
 *    gradient are fp32. All arithmetic is fp32; an output is rounded once, to
 *    nearest even.
 *  - Activations take explicit strides, in elements, outermost first (S, B and,
 *    for the gated norm, H), the last axis adjacent. Strides may be zero and of
 *    any alignment, rows of 16-byte alignment move faster; negative strides are
 *    refused. Weights and every output are dense.
 *  - A single token of each sequence is S = 1.
 *  - Pointers are DEVICE pointers owned by the caller, with the alignment of
 *    their element. Outputs must not overlap inputs or each other. The library
 *    allocates nothing and keeps nothing between calls; what a backward needs
 *    is in `workspace` (16-byte aligned), sized by the *_workspace_size call,
 *    whose contents on entry are ignored.
 *  - Every call enqueues on `stream` of the current device and returns without
 *    waiting. Results are deterministic: no atomics, every sum in an order
 *    that depends on the shape only.
 *  - Limits: 1 <= S <= 2^31 - 4096, 1 <= B <= 65535, 1 <= H <= 2^20, rows
 *    (S*B*H of the gated norm, S*B of the residual norm) below 2^31, and rows
 *    of 1 to 16384 values; eps finite and not negative. Squares are summed in
 *    fp32: rows of values above some 1e18 / sqrt(their number) are past it.
 *
 * Errors as in mcc1d_ssm.h.
 */
#ifndef MCC1D_NORM_H
#define MCC1D_NORM_H

#include <stdint.h>

#include "mcc1d.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Flag of the residual norm: residual, h and their gradients are fp32. */
enum { MCC1D_WIDE = 4 };

/* Required: x, weight, y. flags is 0. */
typedef struct mcc1d_gated_norm_args {
    const void *x;              /* [S,B,H,D] */
    int64_t x_strides[3];       /* S, B, H */
    const void *z;              /* [S,B,H,D] or NULL */
    int64_t z_strides[3];
    const void *weight;         /* [D] */
    void *y;                    /* [S,B,H,D] out */
    int64_t S, B, H, D;
    double eps;
    int32_t dtype, flags;
} mcc1d_gated_norm_args;

int32_t mcc1d_gated_norm(const mcc1d_gated_norm_args *a, void *stream);

/* Its gradients. `fwd` holds the forward's inputs (its y is ignored). Required:
 * grad_y, grad_x, grad_weight; grad_z needs z and may be NULL. */
typedef struct mcc1d_gated_norm_bwd_args {
    mcc1d_gated_norm_args fwd;
    const void *grad_y;         /* [S,B,H,D] */
    int64_t grad_y_strides[3];
    void *grad_x, *grad_z;      /* [S,B,H,D] out */
    void *grad_weight;          /* [D] out */
} mcc1d_gated_norm_bwd_args;

int32_t mcc1d_gated_norm_bwd_workspace_size(const mcc1d_gated_norm_bwd_args *a, uint64_t *bytes_out);
int32_t mcc1d_gated_norm_bwd(const mcc1d_gated_norm_bwd_args *a, void *workspace, uint64_t workspace_bytes,
                             void *stream);

/* Required: x, residual, weight, y, h. flags: MCC1D_WIDE or 0. */
typedef struct mcc1d_residual_norm_args {
    const void *x;              /* [S,B,H] */
    int64_t x_strides[2];       /* S, B */
    const void *residual;       /* [S,B,H] */
    int64_t residual_strides[2];
    const void *weight;         /* [H] */
    const void *post_weight;    /* [H] or NULL */
    const float *scale;         /* [H] or NULL */
    void *y, *h;                /* [S,B,H] out */
    int64_t S, B, H;
    double eps;
    int32_t dtype, flags;
} mcc1d_residual_norm_args;

int32_t mcc1d_residual_norm(const mcc1d_residual_norm_args *a, void *stream);

/* Its gradients, of any loss with gradient grad_y of y and grad_h of h. `fwd`
 * holds the forward's inputs (its y and h are ignored). Required: grad_y,
 * grad_x, grad_residual, grad_weight; grad_post_weight needs post_weight and
 * grad_scale needs scale, and each may be NULL. */
typedef struct mcc1d_residual_norm_bwd_args {
    mcc1d_residual_norm_args fwd;
    const void *grad_y;         /* [S,B,H] */
    int64_t grad_y_strides[2];
    const void *grad_h;         /* [S,B,H] or NULL */
    int64_t grad_h_strides[2];
    void *grad_x, *grad_residual; /* [S,B,H] out */
    void *grad_weight, *grad_post_weight; /* [H] out */
    float *grad_scale;          /* [H] out */
} mcc1d_residual_norm_bwd_args;

int32_t mcc1d_residual_norm_bwd_workspace_size(const mcc1d_residual_norm_bwd_args *a, uint64_t *bytes_out);
int32_t mcc1d_residual_norm_bwd(const mcc1d_residual_norm_bwd_args *a, void *workspace, uint64_t workspace_bytes,
                                void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MCC1D_NORM_H */
