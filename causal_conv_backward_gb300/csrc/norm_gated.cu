// norm_gated.cu - the gated norm and its gradients, and the sums over rows of
// both norms' weights.
#include <algorithm>

#include "norm_common.cuh"

namespace mcc1d {

namespace {

struct GatedParams {
    const void *x, *z, *weight, *grad_y;
    void *y, *grad_x, *grad_z;
    float *part;
    RowAddress xs, zs, gs;
    RowOrder order;
    uint32_t rows;
    int32_t D;
    float eps, inv_D;
};

template <int DT, class R>
__global__ void __launch_bounds__(R::THREADS, 1024 / R::THREADS) mcc1d_norm_gated_fwd(const __grid_constant__ GatedParams p)
{
    __shared__ float shared[2][3][32];
    int turn = 0;
    const uint32_t row = blockIdx.x * R::ROWS + threadIdx.x / R::TPR;
    const bool there = row < p.rows;
    const uint32_t r = there ? row : p.rows - 1;
    float x[R::E], w[R::E], z[R::E];
    const auto xr = load_share<DT, R>(p.x, p.order.at(p.xs, r), p.D);
    Share<DT, R> zr;
    if (p.z)
        zr = load_share<DT, R>(p.z, p.order.at(p.zs, r), p.D);
    load_values<DT, R>(p.weight, 0, p.D, w);
    values<DT, R>(xr, x);
    float s[1] = {0.f};
#pragma unroll
    for (int e = 0; e < R::E; ++e)
        s[0] = fmaf(x[e], x[e], s[0]);
    row_sums<R>(s, &shared, turn);
    const float rms = inverse_root(fmaf(s[0], p.inv_D, p.eps));
#pragma unroll
    for (int e = 0; e < R::E; ++e)
        x[e] = x[e] * rms * w[e];
    if (p.z) {
        values<DT, R>(zr, z);
#pragma unroll
        for (int e = 0; e < R::E; ++e)
            x[e] *= z[e] * sigmoid(z[e]);
    }
    if (there)
        store_values<DT, R>(p.y, (int64_t)row * p.D, p.D, x);
}

// With n = x r, r = 1/rms(x), g = grad_y silu(z):
//   grad_weight = sum of g n over the rows,  grad_z = grad_y n weight silu'(z),
//   grad_x = r (g weight - n mean(g weight n))
template <int DT, class R>
__global__ void __launch_bounds__(R::THREADS, R::THREADS <= 256 ? 768 / R::THREADS : 1) mcc1d_norm_gated_bwd(const __grid_constant__ GatedParams p)
{
    __shared__ float shared[2][3][32];
    __shared__ float joined[R::ROWS > 1 ? R::ROWS * R::TPR * R::E : 1];
    extern __shared__ uint8_t sums[];
    int turn = 0;
    float w[R::E];
    load_values<DT, R>(p.weight, 0, p.D, w);
    typedef Totals<R, 1> Sums;
    Sums gw(sums);
    // rows one ahead of their use
    Share<DT, R> xn, gn, zn;
    const auto ask = [&](uint32_t first) {
        const uint32_t row = first + threadIdx.x / R::TPR, at = row < p.rows ? row : p.rows - 1;
        xn = load_share<DT, R>(p.x, p.order.at(p.xs, at), p.D);
        gn = load_share<DT, R>(p.grad_y, p.order.at(p.gs, at), p.D);
        if (p.z)
            zn = load_share<DT, R>(p.z, p.order.at(p.zs, at), p.D);
    };
    const uint32_t step = gridDim.x * R::ROWS;
    if (Sums::HELD)
        ask(blockIdx.x * R::ROWS);
    for (uint32_t first = blockIdx.x * R::ROWS; first < p.rows; first += step) {
        const uint32_t row = first + threadIdx.x / R::TPR;
        const bool there = row < p.rows;
        float x[R::E], g[R::E];
        if (!Sums::HELD)
            ask(first);
        const Share<DT, R> xr = xn, gr = gn, zr = zn;
        if (Sums::HELD && p.rows - first > step)
            ask(first + step);
        values<DT, R>(xr, x);
        values<DT, R>(gr, g);
        // the gate z sigmoid(z), and grad_y times its derivative
        float gz[R::E];
        if (p.z) {
            float z[R::E];
            values<DT, R>(zr, z);
#pragma unroll
            for (int e = 0; e < R::E; e += 2) {
                const float2 sig = sigmoid2(pair(z, e)), gate = mul2(pair(z, e), sig), one = make_float2(1.f, 1.f);
                put(gz, e, mul2(pair(g, e), fma2(gate, sub2(one, sig), sig)));
                put(g, e, mul2(pair(g, e), gate));
            }
        }
        float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int e = 0; e < R::E; e += 2) {
            s2[0] = fma2(pair(x, e), pair(x, e), s2[0]);
            s2[1] = fma2(mul2(pair(g, e), pair(w, e)), pair(x, e), s2[1]);
        }
        float s[2] = {s2[0].x + s2[0].y, s2[1].x + s2[1].y};
        row_sums<R>(s, &shared, turn);
        const float rms = inverse_root(fmaf(s[0], p.inv_D, p.eps));
        const float along = s[1] * p.inv_D * rms;      // mean(g weight n)
        if (there) {
            const float2 r = make_float2(rms, rms);
#pragma unroll
            for (int e = 0; e < R::E; e += 2) {
                const float2 n = mul2(pair(x, e), r);
                gw.add(0, e, pair(g, e), n);
                put(g, e, mul2(r, fma2(n, make_float2(-along, -along), mul2(pair(g, e), pair(w, e)))));
                put(x, e, n);
            }
            store_values<DT, R>(p.grad_x, (int64_t)row * p.D, p.D, g);
            if (p.grad_z) {
#pragma unroll
                for (int e = 0; e < R::E; e += 2)
                    put(gz, e, mul2(pair(gz, e), mul2(pair(x, e), pair(w, e))));
                store_values<DT, R>(p.grad_z, (int64_t)row * p.D, p.D, gz);
            }
        }
    }
    gw.get(0, w);
    store_part<R>(w, p.part, p.D, &joined);
}

// out[c] = sum of part[p][c]: 32 columns to a block of 8 warps, each warp its
// share of the parts, the warps' sums joined in order.
__global__ void __launch_bounds__(256) mcc1d_norm_sums(const __grid_constant__ ColumnSums s, int32_t parts, int32_t columns)
{
    __shared__ float joined[8][32];
    previous_done();
    if (!s.out[blockIdx.y])
        return;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < columns) {
        const float *part = s.part[blockIdx.y] + c;
        int p = warp;
        for (; p + 24 < parts; p += 32)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                a[k] += part[(int64_t)(p + 8 * k) * columns];
        for (; p < parts; p += 8)
            a[0] += part[(int64_t)p * columns];
    }
    joined[warp][lane] = (a[0] + a[1]) + (a[2] + a[3]);
    __syncthreads();
    if (warp > 0 || c >= columns)
        return;
    float sum = joined[0][lane];
#pragma unroll
    for (int k = 1; k < 8; ++k)
        sum += joined[k][lane];
    if (s.type[blockIdx.y] == 2)
        static_cast<float *>(s.out[blockIdx.y])[c] = sum;
    else
        static_cast<uint16_t *>(s.out[blockIdx.y])[c] =
            (uint16_t)(s.type[blockIdx.y] == 0 ? pack2<0>(make_float2(sum, 0.f)) : pack2<1>(make_float2(sum, 0.f)));
}

GatedParams gated_params(const mcc1d_gated_norm_args &a)
{
    GatedParams p = {};
    p.x = a.x, p.z = a.z, p.weight = a.weight, p.y = a.y;
    p.xs = {a.x_strides[0], a.x_strides[1], a.x_strides[2]};
    p.zs = {a.z_strides[0], a.z_strides[1], a.z_strides[2]};
    p.order.B = Divisor(a.B), p.order.H = Divisor(a.H);
    p.rows = (uint32_t)(a.S * a.B * a.H), p.D = (int32_t)a.D;
    p.eps = (float)a.eps, p.inv_D = (float)(1.0 / (double)a.D);
    return p;
}

bool vectors(const mcc1d_gated_norm_args &a, uintptr_t more, int64_t more_steps)
{
    const int64_t zs = a.z ? a.z_strides[0] | a.z_strides[1] | a.z_strides[2] : 0;
    return vectors_for(a.D, (uintptr_t)a.x | (uintptr_t)a.z | (uintptr_t)a.weight | more,
                       a.x_strides[0] | a.x_strides[1] | a.x_strides[2] | zs | more_steps);
}

}  // namespace

// Blocks of a backward over this many rows: one wave of `threads` to an SM, so
// that the partial sums of D columns stay small beside the rows.
int64_t norm_bwd_blocks(int64_t rows, int64_t columns, bool vec, int threads)
{
    int64_t blocks = 0;
    with_row_shape_bwd(columns, vec, [&](auto shape) {
        typedef decltype(shape) R;
        blocks = std::min<int64_t>((rows + R::ROWS - 1) / R::ROWS, kNumSMs * std::max(1, threads / R::THREADS));
        return 0;
    });
    return blocks;
}

bool gated_norm_vectors(const mcc1d_gated_norm_bwd_args &a)
{
    return vectors(a.fwd, (uintptr_t)a.grad_y | (uintptr_t)a.grad_x | (uintptr_t)a.grad_z,
                   a.grad_y_strides[0] | a.grad_y_strides[1] | a.grad_y_strides[2]);
}

int32_t launch_gated_norm(const mcc1d_gated_norm_args &a, cudaStream_t stream)
{
    const GatedParams p = gated_params(a);
    return with_row_shape(a.D, vectors(a, (uintptr_t)a.y, 0), [&](auto shape) {
        typedef decltype(shape) R;
        const dim3 grid((unsigned)((p.rows + R::ROWS - 1) / R::ROWS));
        return a.dtype == 0 ? launch(mcc1d_norm_gated_fwd<0, R>, grid, R::THREADS, 0, stream, p)
                            : launch(mcc1d_norm_gated_fwd<1, R>, grid, R::THREADS, 0, stream, p);
    });
}

int32_t launch_gated_norm_bwd(const mcc1d_gated_norm_bwd_args &a, float *workspace, cudaStream_t stream)
{
    GatedParams p = gated_params(a.fwd);
    p.grad_y = a.grad_y, p.grad_x = a.grad_x, p.grad_z = a.grad_z, p.part = workspace;
    p.gs = {a.grad_y_strides[0], a.grad_y_strides[1], a.grad_y_strides[2]};
    const bool vec = gated_norm_vectors(a);
    const int64_t blocks = norm_bwd_blocks(p.rows, a.fwd.D, vec, kGatedThreads);
    const int32_t st = with_row_shape_bwd(a.fwd.D, vec, [&](auto shape) {
        typedef decltype(shape) R;
        return a.fwd.dtype == 0 ? launch_totals<R, 1>(mcc1d_norm_gated_bwd<0, R>, blocks, stream, p)
                                : launch_totals<R, 1>(mcc1d_norm_gated_bwd<1, R>, blocks, stream, p);
    });
    if (st != kOk)
        return st;
    const ColumnSums s = {{workspace}, {a.grad_weight}, {a.fwd.dtype}};
    return launch_column_sums(s, blocks, a.fwd.D, 1, stream);
}

int32_t launch_column_sums(const ColumnSums &s, int64_t parts, int64_t columns, int sums, cudaStream_t stream)
{
    return launch_as(true, mcc1d_norm_sums, dim3((unsigned)((columns + 31) / 32), (unsigned)sums), 256, 0, stream, s, (int32_t)parts,
                     (int32_t)columns);
}

}  // namespace mcc1d
