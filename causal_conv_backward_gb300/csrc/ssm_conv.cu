// ssm_conv.cu - the short convolution of a selective state space layer over
// prompts and for single tokens: bias, SiLU, carried windows, lengths.
//
//   pre(t) = bias + sum over k of weight(k) x(t-W+1+k),  y = pre sigmoid(pre)
//
// One thread owns V adjacent channels of one sequence and walks L rows with
// the last W-1 rows in registers, so x is read once but for W-1 rows per L.
// The call moves 4 bytes per element against 2 W + 5 flops and two special
// functions and is bound by memory; the rows travel through a ring in shared
// memory (RowRing), three batches ahead of their use, since registers do not
// hold the bytes that have to be in flight. Measured, bf16, W = 4: 162 us on
// 8192 x 8 x 4096 (0.97 of the measured copy bandwidth), 46 us on
// 4096 x 8 x 2048 (0.85; 57 with eight rows in registers); wider kernels run
// into their arithmetic (W = 8: 62 us); rows aligned to 4 bytes alone take 55 us,
// rows at odd addresses, two bytes per lane, 99.
#include "plan.h"
#include "ssm.h"
#include "ssm_common.cuh"

namespace mcc1d {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = 4;     // rows of a batch
constexpr int kStages = 4;   // batches, all but one in flight

struct ConvParams {
    const uint16_t *x, *weight, *bias, *state;
    const int32_t *lengths;
    uint16_t *y, *final_state;
    int64_t xs, xb, S, B, H, vecs;   // vecs = H / V
    int32_t L, silu;
};

// Row t of a sequence behind its carried window: x for t >= 0, else the
// window's row t + W-1, or zeros without one.
template <int V>
__device__ __forceinline__ Vec<V> window_row(const uint16_t *x, int64_t xs, const uint16_t *state, int64_t H,
                                             int W, int64_t t)
{
    if (t >= 0)
        return vload<V>(x + t * xs);
    return state ? vload<V>(state + (t + W - 1) * H) : vzero<V>();
}

// SILU: with the activation. Single channels (V = 1) take it from p.silu: there
// the branch keeps the next rows' loads ahead of the arithmetic (odd rows,
// 4096 x 8 x 2047: 99 us against 117), elsewhere it keeps rows from
// interleaving.
template <int DT, int V, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) mcc1d_ssm_conv_fwd(const ConvParams p)
{
    constexpr int P = Vec<V>::P;
    using Ring = RowRing<V, 1, kRows, kStages>;
    __shared__ __align__(16) uint8_t slots[V == 1 ? 16 : kThreads * Ring::BYTES_PER_THREAD];
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= p.B * p.vecs)
        return;
    const int64_t b = id / p.vecs, h = (id - b * p.vecs) * V;
    const int64_t t0 = (int64_t)blockIdx.y * p.L, t1 = t0 + p.L < p.S ? t0 + p.L : p.S;
    const int64_t len = clamped_length(p.lengths, b, p.S);
    const int64_t te = t1 < len ? t1 : len;
    const uint16_t *x = p.x + b * p.xb + h;
    const uint16_t *state = p.state ? p.state + b * (W - 1) * p.H + h : nullptr;
    const int64_t ys = p.B * p.H;
    uint16_t *y = p.y + b * p.H + h;

    if (p.final_state && blockIdx.y == 0) {
        uint16_t *fs = p.final_state + b * (W - 1) * p.H + h;
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
            vstore<V>(fs + i * p.H, window_row<V>(x, p.xs, state, p.H, W, len - (W - 1) + i));
    }
    if (t0 < te) {
        float2 w[W][P], win[W > 1 ? W - 1 : 1][P], bias[P];
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
            const Vec<V> r = window_row<V>(x, p.xs, state, p.H, W, t0 - (W - 1) + i);
#pragma unroll
            for (int e = 0; e < P; ++e)
                win[i][e] = unpack2<DT>(r.u[e]);
        }
        auto emit = [&](const Vec<V> &in, uint16_t *to) {
            Vec<V> out;
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 v = unpack2<DT>(in.u[e]);
                float2 s = bias[e];
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    s = fma2(w[k][e], win[k][e], s);
                s = fma2(w[W - 1][e], v, s);
                if (V > 1 ? SILU : p.silu)
                    s = mul2(s, sigmoid2(s));
                out.u[e] = pack2<DT>(s);
#pragma unroll
                for (int k = 0; k < W - 2; ++k)
                    win[k][e] = win[k + 1][e];
                if (W > 1)
                    win[W > 1 ? W - 2 : 0][e] = v;
            }
            vstore<V>(to, out);
        };
        const uint16_t *src = x + t0 * p.xs;
        uint16_t *dst = y + t0 * ys;
        int64_t left = te - t0;
        Ring ring;
        ring.src[0] = src;
        ring.step[0] = p.xs;
        ring.left = left;
        ring.slots = slots;
        ring.threads = kThreads;
        ring.start();
        for (; left >= kRows; left -= kRows) {
            Vec<V> in[kRows];
            ring.take(in);
#pragma unroll
            for (int r = 0; r < kRows; ++r, dst += ys)
                emit(in[r], dst);
        }
        src += (te - t0 - left) * p.xs;
        Vec<V> rest[kRows - 1];
#pragma unroll
        for (int r = 0; r < kRows - 1; ++r, src += p.xs)
            rest[r] = r < left ? vload<V>(src) : vzero<V>();
#pragma unroll
        for (int r = 0; r < kRows - 1; ++r, dst += ys)
            if (r < left)
                emit(rest[r], dst);
    }
    for (int64_t t = t0 > te ? t0 : te; t < t1; ++t)
        vstore<V>(y + t * ys, vzero<V>());
}

struct StepParams {
    const uint16_t *x, *weight, *bias;
    uint16_t *state, *y;
    const int32_t *slots;
    int64_t xb, rows, B, H, vecs;
    int32_t silu;
};

// One token: the window's W-1 rows and x in, y and the moved window out.
template <int DT, int V, int W>
__global__ void __launch_bounds__(kThreads) mcc1d_ssm_conv_step(const StepParams p)
{
    constexpr int P = Vec<V>::P;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= p.B * p.vecs)
        return;
    const int64_t b = id / p.vecs, h = (id - b * p.vecs) * V;
    uint16_t *y = p.y + b * p.H + h;
    const int64_t slot = p.slots ? (int64_t)p.slots[b] : b;
    if (slot < 0 || slot >= p.rows) {
        vstore<V>(y, vzero<V>());
        return;
    }
    uint16_t *state = p.state + slot * (W - 1) * p.H + h;
    Vec<V> row[W], wt[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const uint16_t *src = state + k * p.H;   // written below: not through the read-only path
        if constexpr (V == 8) {
            const uint4 v = *reinterpret_cast<const uint4 *>(src);
            row[k].u[0] = v.x, row[k].u[1] = v.y, row[k].u[2] = v.z, row[k].u[3] = v.w;
        } else {
            row[k].u[0] = *src;
        }
    }
    row[W - 1] = vload<V>(p.x + b * p.xb + h);
#pragma unroll
    for (int k = 0; k < W; ++k)
        wt[k] = vload<V>(p.weight + k * p.H + h);
    const Vec<V> rb = p.bias ? vload<V>(p.bias + h) : vzero<V>();
    Vec<V> out;
#pragma unroll
    for (int e = 0; e < P; ++e) {
        float2 s = unpack2<DT>(rb.u[e]);
#pragma unroll
        for (int k = 0; k < W; ++k)
            s = fma2(unpack2<DT>(wt[k].u[e]), unpack2<DT>(row[k].u[e]), s);
        if (p.silu)
            s = mul2(s, sigmoid2(s));
        out.u[e] = pack2<DT>(s);
    }
    vstore<V>(y, out);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        vstore<V>(state + k * p.H, row[k + 1]);
}

bool aligned(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

template <int DT, bool SILU>
int32_t run_fwd(const ConvParams &p, int V, int W, dim3 grid, cudaStream_t s)
{
    switch (W) {
#define MCC1D_CASE(w)                                                            \
    case w:                                                                      \
        return V == 1 ? launch(mcc1d_ssm_conv_fwd<DT, 1, w, true>, grid, kThreads, 0, s, p)   \
               : V == 2 ? launch(mcc1d_ssm_conv_fwd<DT, 2, w, SILU>, grid, kThreads, 0, s, p) \
                        : launch(mcc1d_ssm_conv_fwd<DT, conv_vec(w), w, SILU>, grid, kThreads, 0, s, p);
        MCC1D_CASE(1) MCC1D_CASE(2) MCC1D_CASE(3) MCC1D_CASE(4)
        MCC1D_CASE(5) MCC1D_CASE(6) MCC1D_CASE(7) MCC1D_CASE(8)
#undef MCC1D_CASE
    }
    return kErrShape;
}

template <int DT, int V>
int32_t run_step(const StepParams &p, int W, dim3 grid, cudaStream_t s)
{
    switch (W) {
#define MCC1D_CASE(w) case w: return launch(mcc1d_ssm_conv_step<DT, V, w>, grid, kThreads, 0, s, p);
        MCC1D_CASE(1) MCC1D_CASE(2) MCC1D_CASE(3) MCC1D_CASE(4)
        MCC1D_CASE(5) MCC1D_CASE(6) MCC1D_CASE(7) MCC1D_CASE(8)
#undef MCC1D_CASE
    }
    return kErrShape;
}

}  // namespace

namespace {

int fwd_vec(const mcc1d_short_conv_args &a)
{
    const uintptr_t any = (uintptr_t)a.x | (uintptr_t)a.weight | (uintptr_t)a.bias | (uintptr_t)a.state |
                          (uintptr_t)a.y | (uintptr_t)a.final_state;
    const int64_t steps = a.H | a.x_strides[0] | a.x_strides[1];
    return conv_vec_for((int)a.W, any, steps);
}

}  // namespace

int32_t launch_short_conv(const mcc1d_short_conv_args &a, cudaStream_t stream)
{
    ConvParams p;
    p.x = (const uint16_t *)a.x;
    p.weight = (const uint16_t *)a.weight;
    p.bias = (const uint16_t *)a.bias;
    p.state = (const uint16_t *)a.state;
    p.lengths = a.lengths;
    p.y = (uint16_t *)a.y;
    p.final_state = (uint16_t *)a.final_state;
    p.xs = a.x_strides[0];
    p.xb = a.x_strides[1];
    p.S = a.S;
    p.B = a.B;
    p.silu = (a.flags & MCC1D_SILU) != 0;
    p.H = a.H;
    const int V = fwd_vec(a);
    p.vecs = a.H / V;
    const int64_t lanes = a.B * p.vecs, blocks = (lanes + kThreads - 1) / kThreads;
    // Long runs of rows re-read fewer window rows; short ones give more threads.
    // 4096 x 8 x 2048: W = 4 48 us with runs of 32 rows, 46 with 128; W = 8 118 and 76.
    int64_t L = 128;
    while (L > 8 && blocks * ((a.S + L - 1) / L) < 152 * 8)
        L /= 2;
    while ((a.S + L - 1) / L > 65535)
        L *= 2;
    p.L = (int32_t)L;
    const dim3 grid((unsigned)blocks, (unsigned)((a.S + L - 1) / L));
    const bool silu = p.silu != 0;
    const auto run = a.dtype == 0 ? (silu ? run_fwd<0, true> : run_fwd<0, false>) : (silu ? run_fwd<1, true> : run_fwd<1, false>);
    return run(p, V, (int)a.W, grid, stream);
}

int32_t launch_short_conv_step(const mcc1d_short_conv_step_args &a, cudaStream_t stream)
{
    StepParams p;
    p.x = (const uint16_t *)a.x;
    p.weight = (const uint16_t *)a.weight;
    p.bias = (const uint16_t *)a.bias;
    p.state = (uint16_t *)a.state;
    p.y = (uint16_t *)a.y;
    p.slots = a.slots;
    p.xb = a.x_stride;
    p.rows = a.cache_rows;
    p.B = a.B;
    p.H = a.H;
    p.silu = (a.flags & MCC1D_SILU) != 0;
    const bool wide = a.H % 8 == 0 && p.xb % 8 == 0 && aligned(a.x, 16) && aligned(a.weight, 16) &&
                      aligned(a.bias, 16) && aligned(a.state, 16) && aligned(a.y, 16);
    p.vecs = a.H / (wide ? 8 : 1);
    const dim3 grid((unsigned)((a.B * p.vecs + kThreads - 1) / kThreads));
    if (a.dtype == 0)
        return wide ? run_step<0, 8>(p, (int)a.W, grid, stream) : run_step<0, 1>(p, (int)a.W, grid, stream);
    return wide ? run_step<1, 8>(p, (int)a.W, grid, stream) : run_step<1, 1>(p, (int)a.W, grid, stream);
}

}  // namespace mcc1d
