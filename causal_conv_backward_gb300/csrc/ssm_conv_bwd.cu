// ssm_conv_bwd.cu - gradients of the short convolution.
//
//   dpre(t)   = grad_y(t) d/dpre [pre sigmoid(pre)],   zero past the length
//   grad_x(t) = sum over j of weight(W-1-j) dpre(t+j)  (+ grad_final_state)
//   grad_weight(k) = sum over b, t of dpre(t) x(t-W+1+k),  grad_bias = sum of dpre
//
// pre is computed again from x rather than kept by the forward: that costs W
// multiply-adds and saves the 2 bytes per element its copy would be read with.
// A warp owns 32 V channels of one sequence and walks L rows, and W-1 more for
// the look-ahead of grad_x, with the last W-1 rows of x and dpre in registers.
// The weight sums stay in registers over the L rows, are added over the
// block's 8 warps in shared memory and over blocks by a second kernel, each in
// a fixed order: nothing depends on scheduling. 6 bytes per element move: bf16,
// W = 4, 8192 x 8 x 4096 takes 289 us (0.82 of the measured copy bandwidth; 779
// with plain loads, 371 with runs of 64 rows, 312 with the activation tested
// per row), 4096 x 8 x 2048 89 us (0.67), with W = 8 152. What is left over
// memory's time is instructions (21 per element) at two blocks of 128 registers
// per SM; at the smaller size it is first of all the 256 blocks, two on 104 of
// the SMs and one on 48.
#include "plan.h"
#include "ssm.h"
#include "ssm_common.cuh"

namespace mcc1d {

namespace {

constexpr int kWarps = 8;
constexpr int kRows = 4;     // rows of a batch
constexpr int kStages = 3;   // batches, all but one in flight
constexpr int kEdge = 2;     // rows that go one by one, loaded together

struct ConvBwdParams {
    const uint16_t *gy, *x, *weight, *bias, *state, *gfs;
    const int32_t *lengths;
    uint16_t *gx, *gstate;
    float *partial;
    int64_t gs, gb, xs, xb, S, B, H, vecs, supers;
    int32_t L, silu;
};

// SILU: with the activation. Single channels (V = 1) take it from p.silu: there
// the branch keeps the next rows' loads ahead of the arithmetic (odd rows,
// 4096 x 8 x 2047: 212 us against 258 when the two were compared, 214 now),
// elsewhere it keeps rows from interleaving.
template <int DT, int V, int W, bool SILU>
__global__ void __launch_bounds__(kWarps * 32, 2) mcc1d_ssm_conv_bwd(const ConvBwdParams p)
{
    constexpr int P = Vec<V>::P;
    constexpr int Wm = W > 1 ? W - 1 : 1;
    using Ring = RowRing<V, 2, kRows, kStages>;
    union Shared {
        uint8_t slots[V == 1 ? 16 : kWarps * 32 * Ring::BYTES_PER_THREAD];
        float2 red[kWarps][W + 1][32][P];      // after the rows
    };
    __shared__ __align__(16) Shared shared;
    next_may_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t vec = (int64_t)blockIdx.x * 32 + lane;
    const int64_t part = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (part >= p.B * p.supers)
        return;
    const int64_t b = part / p.supers, super = part - b * p.supers;
    const bool on = vec < p.vecs;
    const int64_t h = on ? vec * V : 0;
    const int64_t t0 = (super * kWarps + warp) * p.L;
    const int64_t t1 = t0 + p.L < p.S ? t0 + p.L : p.S;

    float2 aw[W + 1][P];    // grad_weight rows, then grad_bias
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e)
            aw[k][e] = make_float2(0.f, 0.f);

    if (on && t0 < p.S) {
        const int64_t len = clamped_length(p.lengths, b, p.S);
        const uint16_t *x = p.x + b * p.xb + h, *gy = p.gy + b * p.gb + h;
        const uint16_t *state = p.state ? p.state + b * (W - 1) * p.H + h : nullptr;
        uint16_t *gx = p.gx + b * p.H + h;
        const int64_t ys = p.B * p.H;
        float2 w[W][P], bias[P], xw[Wm][P], dw[Wm][P];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const Vec<V> r = vload<V>(p.weight + k * p.H + h);
#pragma unroll
            for (int e = 0; e < P; ++e)
                w[k][e] = unpack2<DT>(r.u[e]);
        }
        const Vec<V> rb = p.bias ? vload<V>(p.bias + h) : vzero<V>();
#pragma unroll
        for (int e = 0; e < P; ++e)
            bias[e] = unpack2<DT>(rb.u[e]);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int64_t t = t0 - (W - 1) + i;
            Vec<V> r = vzero<V>();
            if (t >= 0) {
                if (t < len)
                    r = vload<V>(x + t * p.xs);
            } else if (state) {
                r = vload<V>(state + (t + W - 1) * p.H);
            }
#pragma unroll
            for (int e = 0; e < P; ++e) {
                xw[i][e] = unpack2<DT>(r.u[e]);
                dw[i][e] = make_float2(0.f, 0.f);
            }
        }
        // row r gives dpre(r) and, W-1 rows later than its own, grad_x(r-W+1)
        const int64_t rend = t1 + W - 1;
        const int64_t live = rend < len ? rend : len;
        const int64_t first = t0 == 0 ? -(int64_t)(W - 1) : t0;   // first row of grad_x (below 0: the window's)
        // One row: its x and grad_y, `own`: in this run of rows, so counted in the sums; `in`: before the
        // length; gf: the final window's gradient where row r-W+1 of grad_x is in it. Returns grad_x(r-W+1).
        auto row = [&](const Vec<V> &rx, const Vec<V> &rg, const Vec<V> &gf, bool own, bool in) {
            Vec<V> out;
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 v = unpack2<DT>(rx.u[e]);
                float2 d = unpack2<DT>(rg.u[e]);
                if (V > 1 ? SILU : p.silu) {
                    float2 s = bias[e];
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        s = fma2(w[k][e], xw[k][e], s);
                    s = fma2(w[W - 1][e], v, s);
                    // d/ds [s g(s)] = g (1 + s (1 - g)), g the sigmoid
                    const float2 g = sigmoid2(s), one = make_float2(1.f, 1.f);
                    d = mul2(d, mul2(g, fma2(s, fma2(g, make_float2(-1.f, -1.f), one), one)));
                }
                if (!in) {   // an infinite pre, or an infinite x before it, leaves nothing behind
                    d = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        xw[k][e] = make_float2(0.f, 0.f);
                }
                if (own) {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        aw[k][e] = fma2(d, xw[k][e], aw[k][e]);
                    aw[W - 1][e] = fma2(d, v, aw[W - 1][e]);
                    aw[W][e] = add2(aw[W][e], d);
                }
                float2 o = fma2(w[0][e], d, unpack2<DT>(gf.u[e]));
#pragma unroll
                for (int k = W - 2; k >= 0; --k)
                    o = fma2(w[W - 1 - k][e], dw[k][e], o);
                out.u[e] = pack2<DT>(o);
#pragma unroll
                for (int k = 0; k < W - 2; ++k) {
                    xw[k][e] = xw[k + 1][e];
                    dw[k][e] = dw[k + 1][e];
                }
                if (W > 1) {
                    xw[W > 1 ? W - 2 : 0][e] = v;
                    dw[W > 1 ? W - 2 : 0][e] = d;
                }
            }
            return out;
        };
        // Rows r..end-1 with every check, kEdge of them loaded together.
        auto edges = [&](int64_t r, int64_t end) {
            for (; r < end; r += kEdge) {
                Vec<V> ex[kEdge], eg[kEdge], gf[kEdge];
#pragma unroll
                for (int i = 0; i < kEdge; ++i) {
                    const int64_t q = r + i, t = q - (W - 1);
                    const bool in = q < live && q < end;
                    ex[i] = in ? vload<V>(x + q * p.xs) : vzero<V>();
                    eg[i] = in ? vload<V>(gy + q * p.gs) : vzero<V>();
                    gf[i] = vzero<V>();
                    if (p.gfs && t >= len - (W - 1) && t < len && q < end)
                        gf[i] = vload<V>(p.gfs + (b * (W - 1) + (t - (len - (W - 1)))) * p.H + h);
                }
#pragma unroll
                for (int i = 0; i < kEdge; ++i) {
                    const int64_t q = r + i, t = q - (W - 1);
                    if (q >= end)
                        break;
                    const Vec<V> out = row(ex[i], eg[i], gf[i], q < t1, q < live);
                    if (t < first)
                        continue;
                    if (t >= 0)
                        vstore<V>(gx + t * ys, t < len ? out : vzero<V>());   // whatever the weights are
                    else if (p.gstate)
                        vstore<V>(p.gstate + (b * (W - 1) + t + W - 1) * p.H + h, out);
                }
            }
        };
        // the first W-1 rows and what is near the run's or the sequence's end go one by one; between them
        // batches of rows
        int64_t r = t0 + W - 1 < rend ? t0 + W - 1 : rend;
        edges(t0, r);
        const int64_t stop = t1 < len ? t1 : len;
        int64_t left = stop - r;
        uint16_t *to = gx + (r - (W - 1)) * ys;
        Ring ring;
        ring.src[0] = x + r * p.xs;
        ring.src[1] = gy + r * p.gs;
        ring.step[0] = p.xs;
        ring.step[1] = p.gs;
        ring.left = left;
        ring.slots = shared.slots;
        ring.threads = kWarps * 32;
        ring.start();
        for (; left >= kRows; left -= kRows, r += kRows) {
            Vec<V> in[2 * kRows];
            ring.take(in);
            // rows before the final window's: up to W-1 rows before the length no grad_final_state arrives
#pragma unroll
            for (int i = 0; i < kRows; ++i, to += ys)
                vstore<V>(to, row(in[2 * i], in[2 * i + 1], vzero<V>(), true, true));
        }
        edges(r, rend);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e)
            shared.red[warp][k][lane][e] = aw[k][e];
    __syncthreads();
    for (int i = threadIdx.x; i < (W + 1) * 32; i += kWarps * 32) {
        const int k = i / 32, l = i & 31;
        const int64_t v2 = (int64_t)blockIdx.x * 32 + l;
        if (v2 >= p.vecs)
            continue;
        float *out = p.partial + (part * (W + 1) + k) * p.H + v2 * V;
#pragma unroll
        for (int e = 0; e < P; ++e) {
            float2 s = shared.red[0][k][l][e];
#pragma unroll
            for (int q = 1; q < kWarps; ++q)
                s = add2(s, shared.red[q][k][l][e]);
            out[2 * e] = s.x;
            if (V > 1)
                out[2 * e + 1] = s.y;
        }
    }
}

// Sums column i of the [parts][cols] partials: 8 strided runs of parts, then
// the runs in order.
template <int DT>
__global__ void __launch_bounds__(256) mcc1d_ssm_conv_bwd_sum(const float *partial, int64_t parts, int64_t cols,
                                                             int64_t wcols, uint16_t *gw, uint16_t *gbias)
{
    __shared__ float red[8][32];
    previous_done();
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (i < cols)
        for (int64_t r = q; r < parts; r += 8)
            s += partial[r * cols + i];
    red[q][lane] = s;
    __syncthreads();
    if (q == 0 && i < cols) {
#pragma unroll
        for (int k = 1; k < 8; ++k)
            s += red[k][lane];
        const uint16_t v = (uint16_t)pack2<DT>(make_float2(s, 0.f));
        if (i < wcols)
            gw[i] = v;
        else if (gbias)
            gbias[i - wcols] = v;
    }
}

template <int DT, bool SILU>
int32_t run_bwd(const ConvBwdParams &p, int V, int W, dim3 grid, cudaStream_t s)
{
    switch (W) {
#define MCC1D_CASE(w)                                                            \
    case w:                                                                      \
        return V == 1 ? launch(mcc1d_ssm_conv_bwd<DT, 1, w, true>, grid, kWarps * 32, 0, s, p)   \
               : V == 2 ? launch(mcc1d_ssm_conv_bwd<DT, 2, w, SILU>, grid, kWarps * 32, 0, s, p) \
                        : launch(mcc1d_ssm_conv_bwd<DT, conv_vec(w), w, SILU>, grid, kWarps * 32, 0, s, p);
        MCC1D_CASE(1) MCC1D_CASE(2) MCC1D_CASE(3) MCC1D_CASE(4)
        MCC1D_CASE(5) MCC1D_CASE(6) MCC1D_CASE(7) MCC1D_CASE(8)
#undef MCC1D_CASE
    }
    return kErrShape;
}

int bwd_vec(const mcc1d_short_conv_bwd_args &a)
{
    const uintptr_t any = (uintptr_t)a.grad_y | (uintptr_t)a.x | (uintptr_t)a.weight | (uintptr_t)a.bias |
                          (uintptr_t)a.state | (uintptr_t)a.grad_final_state | (uintptr_t)a.grad_x |
                          (uintptr_t)a.grad_state;
    const int64_t steps = a.H | a.grad_y_strides[0] | a.grad_y_strides[1] | a.x_strides[0] | a.x_strides[1];
    return conv_vec_for((int)a.W, any, steps);
}

}  // namespace

ConvBwdPlan conv_bwd_plan(const mcc1d_short_conv_bwd_args &a)
{
    ConvBwdPlan p;
    // Every run of rows begins and ends with rows that go one by one: 64 rows per
    // warp cost 342 us on 8192 x 8 x 4096, 128 310, 256 289 and 512 314. Fewer
    // rows where that leaves less than a block per SM: 4096 x 2 x 2048 takes 33 us
    // with 64 rows (256 blocks), 35 with 128 (128 blocks), 56 with 256. Between
    // one block per SM and two, SMs hold unequal numbers of them and shorter runs
    // do not pay for that: 4096 x 8 x 2048 takes 89 us with 256 rows (256 blocks)
    // and 95 with 128.
    const int64_t wide = (a.H + 127) / 128 * a.B;
    int64_t L = 256;
    while (L > 8 && wide * ((a.S + 8 * L - 1) / (8 * L)) < 152)
        L /= 2;
    p.L = (int32_t)L;
    p.supers = (a.S + kWarps * L - 1) / (kWarps * L);
    p.parts = a.B * p.supers;
    p.bytes = (uint64_t)p.parts * (uint64_t)((a.W + 1) * a.H) * 4u;
    return p;
}

int32_t launch_short_conv_bwd(const mcc1d_short_conv_bwd_args &a, void *workspace, cudaStream_t stream)
{
    const ConvBwdPlan plan = conv_bwd_plan(a);
    ConvBwdParams p;
    p.gy = (const uint16_t *)a.grad_y;
    p.x = (const uint16_t *)a.x;
    p.weight = (const uint16_t *)a.weight;
    p.bias = (const uint16_t *)a.bias;
    p.state = (const uint16_t *)a.state;
    p.gfs = (const uint16_t *)a.grad_final_state;
    p.lengths = a.lengths;
    p.gx = (uint16_t *)a.grad_x;
    p.gstate = (uint16_t *)a.grad_state;
    p.partial = (float *)workspace;
    p.gs = a.grad_y_strides[0];
    p.gb = a.grad_y_strides[1];
    p.xs = a.x_strides[0];
    p.xb = a.x_strides[1];
    p.S = a.S;
    p.B = a.B;
    p.silu = (a.flags & MCC1D_SILU) != 0;
    p.H = a.H;
    p.supers = plan.supers;
    p.L = plan.L;
    const int V = bwd_vec(a);
    p.vecs = a.H / V;
    const int64_t gy = plan.parts < 32768 ? plan.parts : 32768;
    const dim3 grid((unsigned)((p.vecs + 31) / 32), (unsigned)gy, (unsigned)((plan.parts + gy - 1) / gy));
    const bool silu = p.silu != 0;
    const auto run = a.dtype == 0 ? (silu ? run_bwd<0, true> : run_bwd<0, false>) : (silu ? run_bwd<1, true> : run_bwd<1, false>);
    const int32_t st = run(p, V, (int)a.W, grid, stream);
    if (st != kOk)
        return st;
    const int64_t cols = (a.W + 1) * a.H;
    const unsigned blocks = (unsigned)((cols + 31) / 32);
    const auto sum = a.dtype == 0 ? mcc1d_ssm_conv_bwd_sum<0> : mcc1d_ssm_conv_bwd_sum<1>;
    return launch_as(true, sum, blocks, 256, 0, stream, p.partial, plan.parts, cols, a.W * a.H, (uint16_t *)a.grad_weight,
                  (uint16_t *)a.grad_bias);
}

}  // namespace mcc1d
