// norm_residual_bwd.cu - the residual norm's gradients.
//
// With rh = 1/rms(h), q = grad_y weight, the gradient of h is
//   gh = grad_h + rh (q - h rh^2 mean(q h));
// it is grad_residual, and through the branch, gm = gh scale, t = gm post_weight:
//   grad_x = r (t - x r^2 mean(t x)),  or gm without the branch's norm.
// Sums over the rows: grad_weight of grad_y h rh, grad_scale of gh m,
// grad_post_weight of gm x r. h is made again from x and the residual, which
// reads as much as a saved h would and keeps it unrounded.
#include "norm_residual.cuh"

namespace mcc1d {

namespace {

template <int DT, int RT, class R>
__global__ void __launch_bounds__(R::THREADS, R::THREADS <= 512 ? 512 / R::THREADS : 1) mcc1d_norm_residual_bwd(const __grid_constant__ ResidualParams p)
{
    __shared__ float shared[2][3][32];
    __shared__ float joined[R::ROWS > 1 ? R::ROWS * R::TPR * R::E : 1];
    extern __shared__ uint8_t sums[];
    int turn = 0;
    Branch<DT, R> b;
    b.weights(p);
    const auto wr = load_share<DT, R>(p.weight, 0, p.D);
    typedef Totals<R, 3> Sums;      // of weight, post_weight, scale
    Sums total(sums);
    // rows one ahead of their use
    Share<DT, R> xn, gn;
    Share<RT, R> rn, hn;
    const auto ask = [&](uint32_t first) {
        const uint32_t row = first + threadIdx.x / R::TPR, at = row < p.rows ? row : p.rows - 1;
        xn = load_share<DT, R>(p.x, p.order.at(p.xs, at), p.D);
        rn = load_share<RT, R>(p.residual, p.order.at(p.rs, at), p.D);
        gn = load_share<DT, R>(p.grad_y, p.order.at(p.gs, at), p.D);
        if (p.grad_h)
            hn = load_share<RT, R>(p.grad_h, p.order.at(p.ghs, at), p.D);
    };
    const uint32_t step = gridDim.x * R::ROWS;
    if (Sums::HELD)
        ask(blockIdx.x * R::ROWS);
    for (uint32_t first = blockIdx.x * R::ROWS; first < p.rows; first += step) {
        const uint32_t row = first + threadIdx.x / R::TPR;
        const bool there = row < p.rows;
        float x[R::E], h[R::E], g[R::E], w[R::E];
        if (!Sums::HELD)
            ask(first);
        const Share<DT, R> xr = xn, gr = gn;
        const Share<RT, R> rr = rn, hr = hn;
        if (Sums::HELD && p.rows - first > step)
            ask(first + step);
        values<DT, R>(xr, x);
        values<RT, R>(rr, h);
        b.sum(p, x, h, &shared, turn);
        values<DT, R>(gr, g);
        values<DT, R>(wr, w);
        float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < R::E; e += 2) {
            s2[0] = fma2(pair(h, e), pair(h, e), s2[0]);
            s2[1] = fma2(mul2(pair(g, e), pair(w, e)), pair(h, e), s2[1]);
        }
        float s[2] = {s2[0].x + s2[0].y, s2[1].x + s2[1].y};
        row_sums<R>(s, &shared, turn);
        const float rh = inverse_root(fmaf(s[0], p.inv_D, p.eps));
        const float along = s[1] * p.inv_D * rh, in = there ? 1.f : 0.f;      // rows that are not there add nothing
#pragma unroll
        for (int e = 0; e < R::E; e += 2) {
            const float2 n = mul2(pair(h, e), make_float2(rh, rh));
            total.add(0, e, mul2(pair(g, e), make_float2(in, in)), n);
            put(g, e, mul2(make_float2(rh, rh), fma2(n, make_float2(-along, -along), mul2(pair(g, e), pair(w, e)))));
        }
        if (p.grad_h) {
            float gh[R::E];
            values<RT, R>(hr, gh);
#pragma unroll
            for (int e = 0; e < R::E; e += 2)
                put(g, e, add2(pair(g, e), pair(gh, e)));
        }
        if (there)
            store_values<RT, R>(p.grad_residual, (int64_t)row * p.D, p.D, g);
        if (p.scale) {
            float m[R::E], f[R::E];
            b.branch(p, x, m);
            values<2, R>(b.s, f);
#pragma unroll
            for (int e = 0; e < R::E; e += 2) {
                total.add(2, e, mul2(pair(g, e), make_float2(in, in)), pair(m, e));
                put(g, e, mul2(pair(g, e), pair(f, e)));
            }
        }
        if (p.post_weight) {
            float pw[R::E];
            values<DT, R>(b.pw, pw);
            float2 t2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < R::E; e += 2) {
                put(x, e, mul2(pair(x, e), make_float2(b.r, b.r)));
                total.add(1, e, mul2(pair(g, e), make_float2(in, in)), pair(x, e));
                put(g, e, mul2(pair(g, e), pair(pw, e)));
                t2 = fma2(pair(g, e), pair(x, e), t2);
            }
            float t[1] = {t2.x + t2.y};
            row_sums<R>(t, &shared, turn);
            const float back = t[0] * p.inv_D;
#pragma unroll
            for (int e = 0; e < R::E; e += 2)
                put(g, e, mul2(make_float2(b.r, b.r), fma2(pair(x, e), make_float2(-back, -back), pair(g, e))));
        }
        if (there)
            store_values<DT, R>(p.grad_x, (int64_t)row * p.D, p.D, g);
    }
    float *const parts[3] = {p.part, p.part_post, p.part_scale};
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (parts[k]) {
            float x[R::E];
            total.get(k, x);
            store_part<R>(x, parts[k], p.D, &joined);
        }
}

}  // namespace

bool residual_norm_vectors(const mcc1d_residual_norm_bwd_args &a)
{
    return residual_vectors(a.fwd, (uintptr_t)a.grad_y | (uintptr_t)a.grad_h | (uintptr_t)a.grad_x | (uintptr_t)a.grad_residual,
                            a.grad_y_strides[0] | a.grad_y_strides[1] | (a.grad_h ? a.grad_h_strides[0] | a.grad_h_strides[1] : 0));
}

int32_t launch_residual_norm_bwd(const mcc1d_residual_norm_bwd_args &a, float *workspace, cudaStream_t stream)
{
    const mcc1d_residual_norm_args &f = a.fwd;
    ResidualParams p = residual_params(f);
    p.grad_y = a.grad_y, p.grad_h = a.grad_h, p.grad_x = a.grad_x, p.grad_residual = a.grad_residual;
    p.gs = {0, a.grad_y_strides[0], a.grad_y_strides[1]};
    p.ghs = {0, a.grad_h_strides[0], a.grad_h_strides[1]};
    const bool vec = residual_norm_vectors(a);
    const int64_t blocks = norm_bwd_blocks(p.rows, f.H, vec, kResidualThreads);
    p.part = workspace;
    p.part_post = a.grad_post_weight ? workspace + blocks * f.H : nullptr;
    p.part_scale = a.grad_scale ? workspace + 2 * blocks * f.H : nullptr;
    const int32_t st = with_row_shape_bwd(f.H, vec, [&](auto shape) {
        typedef decltype(shape) R;
        const auto go = [&](auto kernel) { return launch_totals<R, 3>(kernel, blocks, stream, p); };
        if (f.flags & MCC1D_WIDE)
            return f.dtype == 0 ? go(mcc1d_norm_residual_bwd<0, 2, R>) : go(mcc1d_norm_residual_bwd<1, 2, R>);
        return f.dtype == 0 ? go(mcc1d_norm_residual_bwd<0, 0, R>) : go(mcc1d_norm_residual_bwd<1, 1, R>);
    });
    if (st != kOk)
        return st;
    const ColumnSums s = {{p.part, p.part_post, p.part_scale}, {a.grad_weight, a.grad_post_weight, a.grad_scale}, {f.dtype, f.dtype, 2}};
    return launch_column_sums(s, blocks, f.H, 3, stream);
}

}  // namespace mcc1d
