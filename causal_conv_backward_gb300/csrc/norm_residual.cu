// norm_residual.cu - the residual norm.
#include "norm_residual.cuh"

namespace mcc1d {

namespace {

// RT: the residual stream's type.
template <int DT, int RT, class R>
__global__ void __launch_bounds__(R::THREADS, 1024 / R::THREADS) mcc1d_norm_residual_fwd(const __grid_constant__ ResidualParams p)
{
    __shared__ float shared[2][3][32];
    int turn = 0;
    const uint32_t row = blockIdx.x * R::ROWS + threadIdx.x / R::TPR;
    const bool there = row < p.rows;
    const uint32_t at = there ? row : p.rows - 1;
    float x[R::E], h[R::E], w[R::E];
    const auto xr = load_share<DT, R>(p.x, p.order.at(p.xs, at), p.D);
    const auto rr = load_share<RT, R>(p.residual, p.order.at(p.rs, at), p.D);
    Branch<DT, R> b;
    b.weights(p);
    values<DT, R>(xr, x);
    values<RT, R>(rr, h);
    b.sum(p, x, h, &shared, turn);
    if (there)
        store_values<RT, R>(p.h, (int64_t)row * p.D, p.D, h);
    load_values<DT, R>(p.weight, 0, p.D, w);
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < R::E; ++e)
        s[0] = fmaf(h[e], h[e], s[0]);
    row_sums<R>(s, &shared, turn);
    const float r = inverse_root(fmaf(s[0], p.inv_D, p.eps));
#pragma unroll
    for (int e = 0; e < R::E; ++e)
        h[e] = h[e] * r * w[e];
    if (there)
        store_values<DT, R>(p.y, (int64_t)row * p.D, p.D, h);
}

}  // namespace

int32_t launch_residual_norm(const mcc1d_residual_norm_args &a, cudaStream_t stream)
{
    const ResidualParams p = residual_params(a);
    return with_row_shape(a.H, residual_vectors(a, (uintptr_t)a.y | (uintptr_t)a.h, 0), [&](auto shape) {
        typedef decltype(shape) R;
        const dim3 grid((unsigned)((p.rows + R::ROWS - 1) / R::ROWS));
        const auto go = [&](auto kernel) { return launch(kernel, grid, R::THREADS, 0, stream, p); };
        if (a.flags & MCC1D_WIDE)
            return a.dtype == 0 ? go(mcc1d_norm_residual_fwd<0, 2, R>) : go(mcc1d_norm_residual_fwd<1, 2, R>);
        return a.dtype == 0 ? go(mcc1d_norm_residual_fwd<0, 0, R>) : go(mcc1d_norm_residual_fwd<1, 1, R>);
    });
}

}  // namespace mcc1d
