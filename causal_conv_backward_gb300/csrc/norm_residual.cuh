// norm_residual.cuh - the residual norm's parameters and their set-up, for the
// forward (norm_residual.cu) and the gradients (norm_residual_bwd.cu).
#pragma once

#include "norm_common.cuh"

namespace mcc1d {

struct ResidualParams {
    const void *x, *residual, *weight, *post_weight, *grad_y, *grad_h;
    const float *scale;
    void *y, *h, *grad_x, *grad_residual;
    float *part, *part_post, *part_scale;     // part_scale and part_post may be null
    RowAddress xs, rs, gs, ghs;
    RowOrder order;
    uint32_t rows;
    int32_t D;
    float eps, inv_D;
};

inline ResidualParams residual_params(const mcc1d_residual_norm_args &a)
{
    ResidualParams p = {};
    p.x = a.x, p.residual = a.residual, p.weight = a.weight, p.post_weight = a.post_weight, p.scale = a.scale;
    p.y = a.y, p.h = a.h;
    // a row of the order is one (s, b): its "heads" are B, its "batch" S
    p.xs = {0, a.x_strides[0], a.x_strides[1]};
    p.rs = {0, a.residual_strides[0], a.residual_strides[1]};
    p.order.B = Divisor(a.S), p.order.H = Divisor(a.B);
    p.rows = (uint32_t)(a.S * a.B), p.D = (int32_t)a.H;
    p.eps = (float)a.eps, p.inv_D = (float)(1.0 / (double)a.H);
    return p;
}

inline bool residual_vectors(const mcc1d_residual_norm_args &a, uintptr_t more, int64_t more_steps)
{
    return vectors_for(a.H,
                       (uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.weight | (uintptr_t)a.post_weight |
                           (uintptr_t)a.scale | more,
                       a.x_strides[0] | a.x_strides[1] | a.residual_strides[0] | a.residual_strides[1] | more_steps);
}

// x -> h, with the branch's own norm and scale: m = x r post_weight.
template <int DT, class R>
struct Branch {
    float r;          // 1 / rms(x), or 1
    Share<2, R> s;
    Share<DT, R> pw;

    __device__ __forceinline__ void weights(const ResidualParams &p)
    {
        if (p.post_weight)
            pw = load_share<DT, R>(p.post_weight, 0, p.D);
        if (p.scale)
            s = load_share<2, R>(p.scale, 0, p.D);
    }
    // h in place of the residual
    __device__ __forceinline__ void sum(const ResidualParams &p, const float (&x)[R::E], float (&h)[R::E], float (*shared)[2][3][32], int &turn)
    {
        r = 1.f;
        if (p.post_weight) {
            float2 v2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < R::E; e += 2)
                v2 = fma2(pair(x, e), pair(x, e), v2);
            float v[1] = {v2.x + v2.y};
            row_sums<R>(v, shared, turn);
            r = inverse_root(fmaf(v[0], p.inv_D, p.eps));
        }
        float m[R::E];
        branch(p, x, m);
        if (p.scale) {
            float f[R::E];
            values<2, R>(s, f);
#pragma unroll
            for (int e = 0; e < R::E; e += 2)
                put(h, e, fma2(pair(m, e), pair(f, e), pair(h, e)));
        } else {
#pragma unroll
            for (int e = 0; e < R::E; e += 2)
                put(h, e, add2(pair(h, e), pair(m, e)));
        }
    }
    // m of x, once r is known
    __device__ __forceinline__ void branch(const ResidualParams &p, const float (&x)[R::E], float (&m)[R::E]) const
    {
        if (p.post_weight) {
            values<DT, R>(pw, m);
#pragma unroll
            for (int e = 0; e < R::E; e += 2)
                put(m, e, mul2(mul2(pair(x, e), make_float2(r, r)), pair(m, e)));
        } else {
#pragma unroll
            for (int e = 0; e < R::E; ++e)
                m[e] = x[e];
        }
    }
};

}  // namespace mcc1d
