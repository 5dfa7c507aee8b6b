// ssm_api.cpp - the extern "C" entry points declared in include/mcc1d_ssm.h.
//
// Checks run in the order null pointers, dtype and flags, shape, strides and
// alignment, workspace, overlap, device; nothing is enqueued before all have passed.
#include <stdint.h>

#include <initializer_list>

#include "checks.h"
#include "device.h"
#include "mcc1d_ssm.h"
#include "plan.h"
#include "ssm.h"

using namespace mcc1d;

namespace {

bool states_ok(int64_t B, int64_t H, int64_t N, int64_t G)
{
    return N >= 1 && N <= kMaxStates && G >= 1 && G <= H && H % G == 0 && B * H <= kMaxGrid / N;
}

Region rows(const void *p, int64_t S, int64_t B, int64_t H, const int64_t (&s)[2])
{
    return Region(p, H, {{S, (uint64_t)s[0]}, {B, (uint64_t)s[1]}});
}
Region rows(const void *p, int64_t B, int64_t H, int64_t stride) { return Region(p, H, {{B, (uint64_t)stride}}); }

int32_t check_apart(const mcc1d_short_conv_args &a)
{
    const int64_t window = 2 * a.B * (a.W - 1) * a.H;
    return apart({{a.y, 2 * a.S * a.B * a.H}, {a.final_state, window}},
                       {rows(a.x, a.S, a.B, a.H, a.x_strides), {a.weight, 2 * a.W * a.H}, {a.bias, 2 * a.H},
                        {a.state, window}, {a.lengths, 4 * a.B}});
}

int32_t check_apart(const mcc1d_short_conv_bwd_args &a, const void *ws, uint64_t bytes)
{
    const int64_t window = 2 * a.B * (a.W - 1) * a.H;
    return apart({{a.grad_x, 2 * a.S * a.B * a.H}, {a.grad_weight, 2 * a.W * a.H}, {a.grad_bias, 2 * a.H},
                        {a.grad_state, window}, {ws, (int64_t)bytes}},
                       {rows(a.grad_y, a.S, a.B, a.H, a.grad_y_strides), rows(a.x, a.S, a.B, a.H, a.x_strides),
                        {a.weight, 2 * a.W * a.H}, {a.bias, 2 * a.H}, {a.state, window}, {a.lengths, 4 * a.B},
                        {a.grad_final_state, window}});
}

int32_t check_apart(const mcc1d_short_conv_step_args &a)
{
    return apart({{a.y, 2 * a.B * a.H}, {a.state, 2 * a.cache_rows * (a.W - 1) * a.H}},
                       {rows(a.x, a.B, a.H, a.x_stride), {a.weight, 2 * a.W * a.H}, {a.bias, 2 * a.H}, {a.slots, 4 * a.B}});
}

// The scan's inputs against these outputs.
int32_t check_apart(const mcc1d_scan_args &a, std::initializer_list<Written> out, const Region &grad_y, const Region &grad_final)
{
    const auto bc = [&](const void *p, const int64_t (&s)[3]) {
        return Region(p, a.N, {{a.S, (uint64_t)s[0]}, {a.B, (uint64_t)s[1]}, {a.G, (uint64_t)s[2]}});
    };
    return apart(out, {rows(a.u, a.S, a.B, a.H, a.u_strides), rows(a.delta, a.S, a.B, a.H, a.delta_strides),
                             rows(a.z, a.S, a.B, a.H, a.z_strides), bc(a.B_, a.B_strides), bc(a.C, a.C_strides),
                             {a.A, 4 * a.H * a.N}, {a.D, 4 * a.H}, {a.delta_bias, 4 * a.H}, {a.state, 4 * a.B * a.H * a.N},
                             {a.lengths, 4 * a.B}, grad_y, grad_final});
}

int32_t check_apart(const mcc1d_scan_args &a, const void *ws, uint64_t bytes)
{
    return check_apart(a, {{a.y, 2 * a.S * a.B * a.H}, {a.final_state, 4 * a.B * a.H * a.N}, {ws, (int64_t)bytes}},
                       {nullptr, 0}, {nullptr, 0});
}

int32_t check_apart(const mcc1d_scan_bwd_args &a, const void *ws, uint64_t bytes)
{
    const mcc1d_scan_args &f = a.fwd;
    const int64_t act = 2 * f.S * f.B * f.H, bc = 2 * f.S * f.B * f.G * f.N, states = 4 * f.B * f.H * f.N;
    return check_apart(f, {{a.grad_u, act}, {a.grad_delta, act}, {a.grad_z, act}, {a.grad_B, bc}, {a.grad_C, bc},
                           {a.grad_A, 4 * f.H * f.N}, {a.grad_D, 4 * f.H}, {a.grad_delta_bias, 4 * f.H},
                           {a.grad_state, states}, {ws, (int64_t)bytes}},
                       rows(a.grad_y, f.S, f.B, f.H, a.grad_y_strides), {a.grad_final_state, states});
}

int32_t check_apart(const mcc1d_scan_step_args &a)
{
    const auto bc = [&](const void *p, const int64_t (&s)[2]) {
        return Region(p, a.N, {{a.B, (uint64_t)s[0]}, {a.G, (uint64_t)s[1]}});
    };
    return apart({{a.y, 2 * a.B * a.H}, {a.state, 4 * a.cache_rows * a.H * a.N}},
                       {rows(a.u, a.B, a.H, a.u_stride), rows(a.delta, a.B, a.H, a.delta_stride),
                        rows(a.z, a.B, a.H, a.z_stride), bc(a.B_, a.B_strides), bc(a.C, a.C_strides), {a.A, 4 * a.H * a.N},
                        {a.D, 4 * a.H}, {a.delta_bias, 4 * a.H}, {a.slots, 4 * a.B}});
}

int32_t check(const mcc1d_short_conv_args *a)
{
    if (!a || !a->x || !a->weight || !a->y)
        return kErrNull;
    if ((a->dtype != 0 && a->dtype != 1) || (a->flags & ~MCC1D_SILU))
        return kErrInvalid;
    if (!shape_ok(a->S, a->B, a->H) || a->W < 1 || a->W > kMaxW)
        return kErrShape;
    if (!strides_ok(a->x_strides) || !on2({a->x, a->weight, a->bias, a->state, a->y, a->final_state}) ||
        !on4({a->lengths}))
        return kErrInvalid;
    return kOk;
}

int32_t check(const mcc1d_short_conv_bwd_args *a)
{
    if (!a || !a->grad_y || !a->x || !a->weight || !a->grad_x || !a->grad_weight)
        return kErrNull;
    if ((a->grad_bias && !a->bias) || (a->grad_state && !a->state))
        return kErrNull;
    if ((a->dtype != 0 && a->dtype != 1) || (a->flags & ~MCC1D_SILU))
        return kErrInvalid;
    if (!shape_ok(a->S, a->B, a->H) || a->W < 1 || a->W > kMaxW)
        return kErrShape;
    if (!strides_ok(a->x_strides) || !strides_ok(a->grad_y_strides) || !on4({a->lengths}) ||
        !on2({a->grad_y, a->x, a->weight, a->bias, a->state, a->grad_final_state, a->grad_x, a->grad_weight,
              a->grad_bias, a->grad_state}))
        return kErrInvalid;
    return conv_bwd_plan(*a).parts <= kMaxGrid / 2 ? kOk : kErrShape;
}

int32_t check(const mcc1d_short_conv_step_args *a)
{
    if (!a || !a->x || !a->weight || !a->y || (!a->state && a->W > 1))
        return kErrNull;
    if ((a->dtype != 0 && a->dtype != 1) || (a->flags & ~MCC1D_SILU))
        return kErrInvalid;
    if (!shape_ok(1, a->B, a->H) || a->W < 1 || a->W > kMaxW || a->cache_rows < 1 ||
        (!a->slots && a->cache_rows < a->B))
        return kErrShape;
    if (a->x_stride < 0 || !on2({a->x, a->state, a->weight, a->bias, a->y}) || !on4({a->slots}))
        return kErrInvalid;
    return kOk;
}

// The scan's inputs; `out`: the forward's own outputs too.
int32_t check(const mcc1d_scan_args *a, bool out)
{
    if (!a || !a->u || !a->delta || !a->B_ || !a->C || !a->A || (out && !a->y))
        return kErrNull;
    if ((a->dtype != 0 && a->dtype != 1) || (a->flags & ~MCC1D_SOFTPLUS))
        return kErrInvalid;
    if (!shape_ok(a->S, a->B, a->H) || !states_ok(a->B, a->H, a->N, a->G))
        return kErrShape;
    if (!strides_ok(a->u_strides) || !strides_ok(a->delta_strides) || (a->z && !strides_ok(a->z_strides)) ||
        !strides_ok(a->B_strides) || !strides_ok(a->C_strides) ||
        !on2({a->u, a->delta, a->z, a->B_, a->C, out ? a->y : nullptr}) ||
        !on4({a->A, a->D, a->delta_bias, a->state, a->lengths, out ? a->final_state : nullptr}))
        return kErrInvalid;
    return kOk;
}

int32_t grid_ok(const ScanPlan &p) { return p.most_blocks <= kMaxGrid ? kOk : kErrShape; }

int32_t check(const mcc1d_scan_bwd_args *a)
{
    if (!a)
        return kErrNull;
    const int32_t st = check(&a->fwd, false);
    if (st != kOk)
        return st;
    if (!a->grad_y || !a->grad_u || !a->grad_delta || !a->grad_A || !a->grad_B || !a->grad_C)
        return kErrNull;
    if ((a->grad_z && !a->fwd.z) || (a->grad_D && !a->fwd.D) || (a->grad_delta_bias && !a->fwd.delta_bias))
        return kErrNull;
    // a thread, of 256 to a block, owns one value of the group sums over [S,B,G] of two padded rows of states
    const mcc1d_scan_args &f = a->fwd;
    if ((double)f.S * (double)f.B * (double)f.G * (2.0 * scan_bwd_plan(*a).np) > (double)(kMaxGrid / 2) * 256.0)
        return kErrShape;
    if (!strides_ok(a->grad_y_strides) ||
        !on2({a->grad_y, a->grad_u, a->grad_delta, a->grad_z, a->grad_B, a->grad_C}) ||
        !on4({a->grad_final_state, a->grad_A, a->grad_D, a->grad_delta_bias, a->grad_state}))
        return kErrInvalid;
    return kOk;
}

int32_t check(const mcc1d_scan_step_args *a)
{
    if (!a || !a->u || !a->delta || !a->B_ || !a->C || !a->A || !a->state || !a->y)
        return kErrNull;
    if ((a->dtype != 0 && a->dtype != 1) || (a->flags & ~MCC1D_SOFTPLUS))
        return kErrInvalid;
    if (!shape_ok(1, a->B, a->H) || !states_ok(a->B, a->H, a->N, a->G) || a->cache_rows < 1 ||
        (!a->slots && a->cache_rows < a->B))
        return kErrShape;
    const int64_t strides[7] = {a->u_stride,     a->delta_stride, a->z ? a->z_stride : 0, a->B_strides[0],
                                a->B_strides[1], a->C_strides[0], a->C_strides[1]};
    for (int64_t s : strides)
        if (s < 0 || s > kMaxGrid)
            return kErrInvalid;
    if ( !on2({a->u, a->delta, a->z, a->B_, a->C, a->y}) ||
        !on4({a->A, a->D, a->delta_bias, a->state, a->slots}))
        return kErrInvalid;
    return kOk;
}

}  // namespace

extern "C" int32_t mcc1d_short_conv(const mcc1d_short_conv_args *a, void *stream)
{
    int32_t st = check(a);
    if (st == kOk)
        st = check_apart(*a);
    if (st == kOk)
        st = check_current_device();
    return st == kOk ? launch_short_conv(*a, static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_short_conv_bwd_workspace_size(const mcc1d_short_conv_bwd_args *a, uint64_t *bytes_out)
{
    if (!bytes_out)
        return kErrNull;
    const int32_t st = check(a);
    if (st == kOk)
        *bytes_out = conv_bwd_plan(*a).bytes;
    return st;
}

extern "C" int32_t mcc1d_short_conv_bwd(const mcc1d_short_conv_bwd_args *a, void *workspace,
                                        uint64_t workspace_bytes, void *stream)
{
    int32_t st = check(a);
    if (st == kOk)
        st = check_workspace(workspace, workspace_bytes, conv_bwd_plan(*a).bytes);
    if (st == kOk)
        st = check_apart(*a, workspace, conv_bwd_plan(*a).bytes);
    if (st == kOk)
        st = check_current_device();
    return st == kOk ? launch_short_conv_bwd(*a, workspace, static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_short_conv_step(const mcc1d_short_conv_step_args *a, void *stream)
{
    int32_t st = check(a);
    if (st == kOk)
        st = check_apart(*a);
    if (st == kOk)
        st = check_current_device();
    return st == kOk ? launch_short_conv_step(*a, static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_scan_workspace_size(const mcc1d_scan_args *a, uint64_t *bytes_out)
{
    if (!bytes_out)
        return kErrNull;
    int32_t st = check(a, true);
    if (st != kOk)
        return st;
    const ScanPlan p = scan_plan(*a);
    st = grid_ok(p);
    if (st == kOk)
        *bytes_out = p.bytes;
    return st;
}

extern "C" int32_t mcc1d_scan(const mcc1d_scan_args *a, void *workspace, uint64_t workspace_bytes, void *stream)
{
    int32_t st = check(a, true);
    if (st != kOk)
        return st;
    const ScanPlan p = scan_plan(*a);
    st = grid_ok(p);
    if (st == kOk)
        st = check_workspace(workspace, workspace_bytes, p.bytes);
    if (st == kOk)
        st = check_apart(*a, workspace, p.bytes);
    if (st == kOk)
        st = check_current_device();
    return st == kOk ? launch_scan(*a, p, workspace, static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_scan_bwd_workspace_size(const mcc1d_scan_bwd_args *a, uint64_t *bytes_out)
{
    if (!bytes_out)
        return kErrNull;
    int32_t st = check(a);
    if (st != kOk)
        return st;
    const ScanPlan p = scan_bwd_plan(*a);
    st = grid_ok(p);
    if (st == kOk)
        *bytes_out = p.bytes;
    return st;
}

extern "C" int32_t mcc1d_scan_bwd(const mcc1d_scan_bwd_args *a, void *workspace, uint64_t workspace_bytes,
                                  void *stream)
{
    int32_t st = check(a);
    if (st != kOk)
        return st;
    const ScanPlan p = scan_bwd_plan(*a);
    st = grid_ok(p);
    if (st == kOk)
        st = check_workspace(workspace, workspace_bytes, p.bytes);
    if (st == kOk)
        st = check_apart(*a, workspace, p.bytes);
    if (st == kOk)
        st = check_current_device();
    return st == kOk ? launch_scan_bwd(*a, p, workspace, static_cast<cudaStream_t>(stream)) : st;
}

extern "C" int32_t mcc1d_scan_step(const mcc1d_scan_step_args *a, void *stream)
{
    int32_t st = check(a);
    if (st == kOk)
        st = check_apart(*a);
    if (st == kOk)
        st = check_current_device();
    return st == kOk ? launch_scan_step(*a, static_cast<cudaStream_t>(stream)) : st;
}
