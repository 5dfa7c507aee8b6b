// norm_api.cpp - the extern "C" entry points declared in include/mcc1d_norm.h.
//
// Checks run in the order null pointers, dtype and flags, shape, strides and
// alignment, workspace, overlap, device; nothing is enqueued before all have passed.
#include <cmath>

#include "checks.h"
#include "device.h"
#include "mcc1d_norm.h"
#include "norm.h"

using namespace mcc1d;

namespace {

bool eps_ok(double eps) { return std::isfinite(eps) && eps >= 0 && eps <= 3e38; }

int32_t check(const mcc1d_gated_norm_args *a, bool out)
{
    if (!a || !a->x || !a->weight || (out && !a->y))
        return kErrNull;
    if ((a->dtype != 0 && a->dtype != 1) || a->flags || !eps_ok(a->eps))
        return kErrInvalid;
    if (!shape_ok(a->S, a->B, a->H) || a->D < 1 || a->D > kMaxNormRow || a->B * a->H > kMaxGrid / a->S)
        return kErrShape;
    if (!strides_ok(a->x_strides) || (a->z && !strides_ok(a->z_strides)) || !on2({a->x, a->z, a->weight, out ? a->y : nullptr}))
        return kErrInvalid;
    return kOk;
}

int32_t check(const mcc1d_gated_norm_bwd_args *a)
{
    if (!a)
        return kErrNull;
    const int32_t st = check(&a->fwd, false);
    if (st != kOk)
        return st;
    if (!a->grad_y || !a->grad_x || !a->grad_weight || (a->grad_z && !a->fwd.z))
        return kErrNull;
    if (!strides_ok(a->grad_y_strides) || !on2({a->grad_y, a->grad_x, a->grad_z, a->grad_weight}))
        return kErrInvalid;
    return kOk;
}

int32_t check(const mcc1d_residual_norm_args *a, bool out)
{
    if (!a || !a->x || !a->residual || !a->weight || (out && (!a->y || !a->h)))
        return kErrNull;
    if ((a->dtype != 0 && a->dtype != 1) || (a->flags & ~MCC1D_WIDE) || !eps_ok(a->eps))
        return kErrInvalid;
    if (!shape_ok(a->S, a->B, a->H) || a->H > kMaxNormRow || a->B > kMaxGrid / a->S)
        return kErrShape;
    const bool wide = (a->flags & MCC1D_WIDE) != 0;
    if (!strides_ok(a->x_strides) || !strides_ok(a->residual_strides) || !on2({a->x, a->weight, a->post_weight, out ? a->y : nullptr}) ||
        !on4({a->scale}) || !(wide ? on4({a->residual, out ? a->h : nullptr}) : on2({a->residual, out ? a->h : nullptr})))
        return kErrInvalid;
    return kOk;
}

int32_t check(const mcc1d_residual_norm_bwd_args *a)
{
    if (!a)
        return kErrNull;
    const int32_t st = check(&a->fwd, false);
    if (st != kOk)
        return st;
    if (!a->grad_y || !a->grad_x || !a->grad_residual || !a->grad_weight || (a->grad_post_weight && !a->fwd.post_weight) ||
        (a->grad_scale && !a->fwd.scale))
        return kErrNull;
    const bool wide = (a->fwd.flags & MCC1D_WIDE) != 0;
    if (!strides_ok(a->grad_y_strides) || (a->grad_h && !strides_ok(a->grad_h_strides)) ||
        !on2({a->grad_y, a->grad_x, a->grad_weight, a->grad_post_weight}) || !on4({a->grad_scale}) ||
        !(wide ? on4({a->grad_h, a->grad_residual}) : on2({a->grad_h, a->grad_residual})))
        return kErrInvalid;
    return kOk;
}

Region heads(const void *p, const mcc1d_gated_norm_args &a, const int64_t (&s)[3])
{
    return Region(p, a.D, {{a.S, (uint64_t)s[0]}, {a.B, (uint64_t)s[1]}, {a.H, (uint64_t)s[2]}});
}

Region rows(const void *p, const mcc1d_residual_norm_args &a, const int64_t (&s)[2], int size)
{
    return Region(p, a.H, {{a.S, (uint64_t)s[0]}, {a.B, (uint64_t)s[1]}}, size);
}

int stream_size(const mcc1d_residual_norm_args &a) { return a.flags & MCC1D_WIDE ? 4 : 2; }

int32_t check_apart(const mcc1d_gated_norm_args &a)
{
    return apart({{a.y, 2 * a.S * a.B * a.H * a.D}}, {heads(a.x, a, a.x_strides), heads(a.z, a, a.z_strides), {a.weight, 2 * a.D}});
}

int32_t check_apart(const mcc1d_gated_norm_bwd_args &a, const void *ws, uint64_t bytes)
{
    const mcc1d_gated_norm_args &f = a.fwd;
    const int64_t act = 2 * f.S * f.B * f.H * f.D;
    return apart({{a.grad_x, act}, {a.grad_z, act}, {a.grad_weight, 2 * f.D}, {ws, (int64_t)bytes}},
                 {heads(f.x, f, f.x_strides), heads(f.z, f, f.z_strides), {f.weight, 2 * f.D}, heads(a.grad_y, f, a.grad_y_strides)});
}

int32_t check_apart(const mcc1d_residual_norm_args &a)
{
    const int64_t n = a.S * a.B * a.H, size = stream_size(a);
    return apart({{a.y, 2 * n}, {a.h, size * n}},
                 {rows(a.x, a, a.x_strides, 2), rows(a.residual, a, a.residual_strides, (int)size), {a.weight, 2 * a.H},
                  {a.post_weight, 2 * a.H}, {a.scale, 4 * a.H}});
}

int32_t check_apart(const mcc1d_residual_norm_bwd_args &a, const void *ws, uint64_t bytes)
{
    const mcc1d_residual_norm_args &f = a.fwd;
    const int64_t n = f.S * f.B * f.H, size = stream_size(f);
    return apart({{a.grad_x, 2 * n}, {a.grad_residual, size * n}, {a.grad_weight, 2 * f.H}, {a.grad_post_weight, 2 * f.H},
                  {a.grad_scale, 4 * f.H}, {ws, (int64_t)bytes}},
                 {rows(f.x, f, f.x_strides, 2), rows(f.residual, f, f.residual_strides, (int)size), {f.weight, 2 * f.H},
                  {f.post_weight, 2 * f.H}, {f.scale, 4 * f.H}, rows(a.grad_y, f, a.grad_y_strides, 2),
                  rows(a.grad_h, f, a.grad_h_strides, (int)size)});
}

uint64_t bytes_of(const mcc1d_gated_norm_bwd_args &a)
{
    const int64_t rows = a.fwd.S * a.fwd.B * a.fwd.H;
    return norm_bwd_bytes(norm_bwd_blocks(rows, a.fwd.D, gated_norm_vectors(a), kGatedThreads), a.fwd.D, 1);
}

uint64_t bytes_of(const mcc1d_residual_norm_bwd_args &a)
{
    return norm_bwd_bytes(norm_bwd_blocks(a.fwd.S * a.fwd.B, a.fwd.H, residual_norm_vectors(a), kResidualThreads), a.fwd.H, 3);
}

template <class A>
int32_t size_of(const A *a, uint64_t *bytes_out)
{
    if (!bytes_out)
        return kErrNull;
    const int32_t st = check(a);
    if (st == kOk)
        *bytes_out = bytes_of(*a);
    return st;
}

template <class A>
int32_t ready(const A *a, const void *workspace, uint64_t workspace_bytes)
{
    int32_t st = check(a);
    if (st == kOk)
        st = check_workspace(workspace, workspace_bytes, bytes_of(*a));
    if (st == kOk)
        st = check_apart(*a, workspace, bytes_of(*a));
    return st == kOk ? check_current_device() : st;
}

template <class A>
int32_t ready(const A *a)
{
    int32_t st = check(a, true);
    if (st == kOk)
        st = check_apart(*a);
    return st == kOk ? check_current_device() : st;
}

}  // namespace

extern "C" int32_t mcc1d_gated_norm(const mcc1d_gated_norm_args *a, void *stream)
{
    const int32_t st = ready(a);
    return st == kOk ? launch_gated_norm(*a, static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_gated_norm_bwd_workspace_size(const mcc1d_gated_norm_bwd_args *a, uint64_t *bytes_out)
{
    return size_of(a, bytes_out);
}

extern "C" int32_t mcc1d_gated_norm_bwd(const mcc1d_gated_norm_bwd_args *a, void *workspace, uint64_t workspace_bytes, void *stream)
{
    const int32_t st = ready(a, workspace, workspace_bytes);
    return st == kOk ? launch_gated_norm_bwd(*a, static_cast<float *>(workspace), static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_residual_norm(const mcc1d_residual_norm_args *a, void *stream)
{
    const int32_t st = ready(a);
    return st == kOk ? launch_residual_norm(*a, static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_residual_norm_bwd_workspace_size(const mcc1d_residual_norm_bwd_args *a, uint64_t *bytes_out)
{
    return size_of(a, bytes_out);
}

extern "C" int32_t mcc1d_residual_norm_bwd(const mcc1d_residual_norm_bwd_args *a, void *workspace, uint64_t workspace_bytes, void *stream)
{
    const int32_t st = ready(a, workspace, workspace_bytes);
    return st == kOk ? launch_residual_norm_bwd(*a, static_cast<float *>(workspace), static_cast<cudaStream_t>(stream)) : st;
}
