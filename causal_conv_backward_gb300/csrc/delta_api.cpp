// delta_api.cpp - the extern "C" entry points declared in include/mcc1d_delta.h.
//
// Checks run in the order null pointers, dtype and flags, shape, strides and
// alignment, workspace, overlap, device; nothing is enqueued before all have passed.
#include <cmath>

#include "checks.h"
#include "delta.h"
#include "device.h"
#include "mcc1d_delta.h"

using namespace mcc1d;

namespace {

constexpr int32_t kFlags = MCC1D_SOFTPLUS | MCC1D_SIGMOID | MCC1D_QK_NORM;

bool heads_ok(int64_t B, int64_t H, int64_t G, int64_t K, int64_t V)
{
    return G >= 1 && G <= H && H % G == 0 && K >= 1 && K <= kMaxKey && V >= 1 && V <= kMaxValue && B * H <= kMaxGrid / (K * V);
}

// The inputs; `out`: the forward's own outputs too.
int32_t check(const mcc1d_delta_args *a, bool out)
{
    if (!a || !a->q || !a->k || !a->v || !a->beta || (a->delta && !a->A) || (out && !a->y))
        return kErrNull;
    if ((a->dtype != 0 && a->dtype != 1) || (a->flags & ~kFlags) || !std::isfinite((float)a->scale))
        return kErrInvalid;
    if (!shape_ok(a->S, a->B, a->H) || !heads_ok(a->B, a->H, a->G, a->K, a->V))
        return kErrShape;
    if (!strides_ok(a->q_strides) || !strides_ok(a->k_strides) || !strides_ok(a->v_strides) || (a->delta && !strides_ok(a->delta_strides)) ||
        !strides_ok(a->beta_strides) || !on2({a->q, a->k, a->v, a->delta, a->beta, out ? a->y : nullptr}) ||
        !on4({a->A, a->delta_bias, a->state, a->lengths, out ? a->final_state : nullptr}))
        return kErrInvalid;
    // blocks are chunks of sequences and heads
    return (double)((a->S + kChunk - 1) / kChunk) * (double)a->B * (double)a->H <= (double)kMaxGrid ? kOk : kErrShape;
}

int32_t check(const mcc1d_delta_bwd_args *a)
{
    if (!a)
        return kErrNull;
    const int32_t st = check(&a->fwd, false);
    if (st != kOk)
        return st;
    const mcc1d_delta_args &f = a->fwd;
    if (!a->grad_y || !a->grad_q || !a->grad_k || !a->grad_v || !a->grad_beta || (f.delta && (!a->grad_delta || !a->grad_A)) ||
        (a->grad_delta && !f.delta) || (a->grad_A && !f.delta) || (a->grad_delta_bias && (!f.delta || !f.delta_bias)))
        return kErrNull;
    if (!strides_ok(a->grad_y_strides) || !on2({a->grad_y, a->grad_q, a->grad_k, a->grad_v, a->grad_delta, a->grad_beta}) ||
        !on4({a->grad_final_state, a->grad_A, a->grad_delta_bias, a->grad_state}))
        return kErrInvalid;
    return kOk;
}

int32_t check(const mcc1d_delta_step_args *a)
{
    if (!a || !a->q || !a->k || !a->v || !a->beta || (a->delta && !a->A) || !a->state || !a->y)
        return kErrNull;
    if ((a->dtype != 0 && a->dtype != 1) || (a->flags & ~kFlags) || !std::isfinite((float)a->scale))
        return kErrInvalid;
    if (!shape_ok(1, a->B, a->H) || !heads_ok(a->B, a->H, a->G, a->K, a->V) || a->cache_rows < 1 || (!a->slots && a->cache_rows < a->B))
        return kErrShape;
    if (!strides_ok(a->q_strides) || !strides_ok(a->k_strides) || !strides_ok(a->v_strides) || (a->delta && a->delta_stride < 0) ||
        a->beta_stride < 0 || !on2({a->q, a->k, a->v, a->delta, a->beta, a->y}) || !on4({a->A, a->delta_bias, a->state, a->slots}))
        return kErrInvalid;
    return kOk;
}

typedef Region::Axis Axis;

Region of(const void *p, int64_t n, std::initializer_list<Axis> axes) { return Region(p, n, axes); }

Axis axis(int64_t count, int64_t step) { return {count, (uint64_t)step}; }

int32_t check_apart(const mcc1d_delta_args &a, std::initializer_list<Written> out, const Region &grad_y, const Region &grad_final)
{
    const auto three = [&](const void *p, int64_t heads, int64_t n, const int64_t (&s)[3]) {
        return of(p, n, {axis(a.S, s[0]), axis(a.B, s[1]), axis(heads, s[2])});
    };
    const auto two = [&](const void *p, const int64_t (&s)[2]) { return of(p, a.H, {axis(a.S, s[0]), axis(a.B, s[1])}); };
    return apart(out, {three(a.q, a.G, a.K, a.q_strides), three(a.k, a.G, a.K, a.k_strides), three(a.v, a.H, a.V, a.v_strides),
                       two(a.delta, a.delta_strides), two(a.beta, a.beta_strides), {a.A, 4 * a.H}, {a.delta_bias, 4 * a.H},
                       {a.state, 4 * a.B * a.H * a.V * a.K}, {a.lengths, 4 * a.B}, grad_y, grad_final});
}

int32_t check_apart(const mcc1d_delta_args &a, const void *ws, uint64_t bytes)
{
    return check_apart(a, {{a.y, 2 * a.S * a.B * a.H * a.V}, {a.final_state, 4 * a.B * a.H * a.V * a.K}, {ws, (int64_t)bytes}},
                       {nullptr, 0}, {nullptr, 0});
}

int32_t check_apart(const mcc1d_delta_bwd_args &a, const void *ws, uint64_t bytes)
{
    const mcc1d_delta_args &f = a.fwd;
    const int64_t t = 2 * f.S * f.B, states = 4 * f.B * f.H * f.V * f.K;
    return check_apart(f, {{a.grad_q, t * f.G * f.K}, {a.grad_k, t * f.G * f.K}, {a.grad_v, t * f.H * f.V}, {a.grad_delta, t * f.H},
                           {a.grad_beta, t * f.H}, {a.grad_A, 4 * f.H}, {a.grad_delta_bias, 4 * f.H}, {a.grad_state, states},
                           {ws, (int64_t)bytes}},
                       of(a.grad_y, f.V, {axis(f.S, a.grad_y_strides[0]), axis(f.B, a.grad_y_strides[1]), axis(f.H, a.grad_y_strides[2])}),
                       {a.grad_final_state, states});
}

int32_t check_apart(const mcc1d_delta_step_args &a)
{
    const auto two = [&](const void *p, int64_t heads, int64_t n, const int64_t (&s)[2]) {
        return of(p, n, {axis(a.B, s[0]), axis(heads, s[1])});
    };
    return apart({{a.y, 2 * a.B * a.H * a.V}, {a.state, 4 * a.cache_rows * a.H * a.V * a.K}},
                 {two(a.q, a.G, a.K, a.q_strides), two(a.k, a.G, a.K, a.k_strides), two(a.v, a.H, a.V, a.v_strides),
                  of(a.delta, a.H, {axis(a.B, a.delta_stride)}), of(a.beta, a.H, {axis(a.B, a.beta_stride)}), {a.A, 4 * a.H},
                  {a.delta_bias, 4 * a.H}, {a.slots, 4 * a.B}});
}

}  // namespace

extern "C" int32_t mcc1d_delta_workspace_size(const mcc1d_delta_args *a, uint64_t *bytes_out)
{
    if (!bytes_out)
        return kErrNull;
    const int32_t st = check(a, true);
    if (st == kOk)
        *bytes_out = delta_plan(*a, false).bytes;
    return st;
}

extern "C" int32_t mcc1d_delta(const mcc1d_delta_args *a, void *workspace, uint64_t workspace_bytes, void *stream)
{
    int32_t st = check(a, true);
    if (st != kOk)
        return st;
    const uint64_t bytes = delta_plan(*a, false).bytes;
    st = check_workspace(workspace, workspace_bytes, bytes);
    if (st == kOk)
        st = check_apart(*a, workspace, bytes);
    if (st == kOk)
        st = check_current_device();
    return st == kOk ? launch_delta(*a, workspace, static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_delta_bwd_workspace_size(const mcc1d_delta_bwd_args *a, uint64_t *bytes_out)
{
    if (!bytes_out)
        return kErrNull;
    const int32_t st = check(a);
    if (st == kOk)
        *bytes_out = delta_bwd_plan(*a).bytes;
    return st;
}

extern "C" int32_t mcc1d_delta_bwd(const mcc1d_delta_bwd_args *a, void *workspace, uint64_t workspace_bytes, void *stream)
{
    int32_t st = check(a);
    if (st != kOk)
        return st;
    const uint64_t bytes = delta_bwd_plan(*a).bytes;
    st = check_workspace(workspace, workspace_bytes, bytes);
    if (st == kOk)
        st = check_apart(*a, workspace, bytes);
    if (st == kOk)
        st = check_current_device();
    return st == kOk ? launch_delta_bwd(*a, workspace, static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_delta_step(const mcc1d_delta_step_args *a, void *stream)
{
    int32_t st = check(a);
    if (st == kOk)
        st = check_apart(*a);
    if (st == kOk)
        st = check_current_device();
    return st == kOk ? launch_delta_step(*a, static_cast<cudaStream_t>(stream)) : st;
}
