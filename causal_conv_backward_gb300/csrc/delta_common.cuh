// delta_common.cuh - what the gated delta rule's kernels share: parameters,
// the gates of a token, and vectors of q and k divided by their lengths.
#pragma once

#include "delta.h"
#include "norm_common.cuh"

namespace mcc1d {

struct DeltaParams {
    const uint16_t *q, *k, *v, *delta, *beta, *grad_y;
    const float *A, *delta_bias, *state, *grad_final;
    const int32_t *lengths;
    uint16_t *y, *grad_v;
    float *final_state, *grad_state;
    int64_t q_s[3], k_s[3], v_s[3], delta_s[2], beta_s[2], gy_s[3];
    int64_t S;
    int32_t B, H, G, K, V;
    float scale;
    int32_t flags;
    DeltaKept kept;
};

inline DeltaParams delta_params(const mcc1d_delta_args &a)
{
    DeltaParams p = {};
    p.q = static_cast<const uint16_t *>(a.q), p.k = static_cast<const uint16_t *>(a.k), p.v = static_cast<const uint16_t *>(a.v);
    p.delta = static_cast<const uint16_t *>(a.delta), p.beta = static_cast<const uint16_t *>(a.beta);
    p.A = a.A, p.delta_bias = a.delta ? a.delta_bias : nullptr, p.state = a.state, p.lengths = a.lengths;
    p.y = static_cast<uint16_t *>(a.y), p.final_state = a.final_state;
    for (int i = 0; i < 3; ++i)
        p.q_s[i] = a.q_strides[i], p.k_s[i] = a.k_strides[i], p.v_s[i] = a.v_strides[i];
    for (int i = 0; i < 2; ++i)
        p.delta_s[i] = a.delta_strides[i], p.beta_s[i] = a.beta_strides[i];
    p.S = a.S, p.B = (int32_t)a.B, p.H = (int32_t)a.H, p.G = (int32_t)a.G, p.K = (int32_t)a.K, p.V = (int32_t)a.V;
    p.scale = (float)a.scale, p.flags = a.flags;
    return p;
}

// The log2 of one decay as the chunks take it, and 2^x for sums of them, no more than
// 2^127. By comparisons, not by the smaller and larger of two: a NaN stays one.
__device__ __forceinline__ float held_log2(float x) { return x < -255.f ? -255.f : x > 255.f ? 255.f : x; }
__device__ __forceinline__ float ex2_held(float x) { return ex2(x > 127.f ? 127.f : x); }

// One 16-bit value.
template <int DT>
__device__ __forceinline__ float value(const uint16_t *p) { return unpack2<DT>(__ldg(p)).x; }

// A token's gates from its raw delta and beta.
struct Gates {
    float raw, dt, log2a, b;    // log2 of the decay
};
__device__ __forceinline__ Gates gates_of(int flags, bool decays, float delta, float bias, float A, float beta)
{
    Gates g;
    g.raw = delta + bias;
    g.dt = flags & MCC1D_SOFTPLUS ? softplus(g.raw) : g.raw;
    g.log2a = decays ? g.dt * (A * kLog2e) : 0.f;
    g.b = flags & MCC1D_SIGMOID ? sigmoid(beta) : beta;
    return g;
}

// 2^x for a decay that a state is multiplied by again and again, token after token
// or chunk after chunk: a bias of its last bit would add up where rounding cancels.
// ex2.approx is low by 0.6e-8 on average at exponents of -1e-5 to -1e-3, by 2e-8 at
// -0.01 to -1, so that no shift of the exponent suits both (3000 steps left a state
// 1.7e-5 too small, with the scan's shift 2.5e-5 too large). This is the exponential
// series of f ln 2 for the f of -1/2..1/2 beside a whole power, off by 5e-9 at its
// end, and 1 exactly for x = 0. NaN stays NaN, and what fp32 cannot hold is 0 or
// infinity.
__device__ __forceinline__ float decay_of(float x)
{
    if (x < -126.f)
        return 0.f;
    if (x >= 128.f)
        return INFINITY;
    const float n = fminf(rintf(x), 127.f), f = x - n;
    float r = 1.5252734e-5f;          // (ln 2)^7 / 7!, and so on
    r = fmaf(r, f, 1.5403530e-4f);
    r = fmaf(r, f, 1.3333558e-3f);
    r = fmaf(r, f, 9.6181291e-3f);
    r = fmaf(r, f, 5.5504109e-2f);
    r = fmaf(r, f, 2.4022651e-1f);
    r = fmaf(r, f, 6.9314718e-1f);
    return fmaf(r, f, 1.f) * __uint_as_float((uint32_t)((int)n + 127) << 23);
}

// What q or k is multiplied by, from its squared length.
__device__ __forceinline__ float unit_factor(int flags, float squares)
{
    return flags & MCC1D_QK_NORM ? inverse_root(squares + (float)kUnitEps) : 1.f;
}

}  // namespace mcc1d
