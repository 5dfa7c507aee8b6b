// delta_tokens.cu - the gated delta rule over prompts token by token, forwards
// and, for the gradients, backwards.
//
// The states stay in registers: eight lanes share a row of K values, a warp has
// 16 rows. Tokens come in groups of kGroup through shared memory, where q and k
// lie divided by their lengths. A token is a chain of two sums over eight lanes and
// an update, which bounds the kernel: 31 tokens of 8 x 16 heads of 128 x 128 take
// 30 us, 0.9 a token; the states alone would take 2.5.
#include "delta_common.cuh"

namespace mcc1d {

namespace {

constexpr int kGroup = 16, kWarps = 4, kRR = 4, kRowsPerBlock = kWarps * 4 * kRR;

template <int KP>
struct TokenShared {
    float q[kGroup][KP], k[kGroup][KP];
    float w[kGroup][kRowsPerBlock];      // v, or grad_y
    float a[kGroup], b[kGroup], kq[kGroup];
};

// Tokens t0.. of sequence b into shared memory (n of them, those past it as
// zeros with a decay of 1).
template <int DT, int KP>
__device__ __forceinline__ void stage(const DeltaParams &p, TokenShared<KP> &s, const uint16_t *w, const int64_t (&w_s)[3], int b, int h,
                                      int row0, int64_t t0, int n)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = h / (p.H / p.G);
    for (int i = warp; i < kGroup; i += kWarps) {
        const int64_t t = t0 + i;
        const bool live = i < n;
        const uint16_t *qp = p.q + t * p.q_s[0] + b * p.q_s[1] + g * p.q_s[2];
        const uint16_t *kp = p.k + t * p.k_s[0] + b * p.k_s[1] + g * p.k_s[2];
        float q[KP / 32], k[KP / 32], sums[3] = {0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
            const int at = j * 32 + lane;
            q[j] = live && at < p.K ? value<DT>(qp + at) : 0.f;
            k[j] = live && at < p.K ? value<DT>(kp + at) : 0.f;
            sums[0] = fmaf(q[j], q[j], sums[0]);
            sums[1] = fmaf(k[j], k[j], sums[1]);
            sums[2] = fmaf(q[j], k[j], sums[2]);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2)
#pragma unroll
            for (int j = 0; j < 3; ++j)
                sums[j] += __shfl_xor_sync(0xFFFFFFFFu, sums[j], d);
        const float fq = unit_factor(p.flags, sums[0]) * p.scale, fk = unit_factor(p.flags, sums[1]);
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
            s.q[i][j * 32 + lane] = q[j] * fq;
            s.k[i][j * 32 + lane] = k[j] * fk;
        }
        const uint16_t *wp = w + t * w_s[0] + b * w_s[1] + h * w_s[2];
        for (int j = lane; j < kRowsPerBlock; j += 32)
            s.w[i][j] = live && row0 + j < p.V ? value<DT>(wp + row0 + j) : 0.f;
        if (lane == 0) {
            Gates gate = {0.f, 0.f, 0.f, 0.f};
            if (live)
                gate = gates_of(p.flags, p.delta != nullptr, p.delta ? value<DT>(p.delta + t * p.delta_s[0] + b * p.delta_s[1] + h) : 0.f,
                                p.delta_bias ? __ldg(p.delta_bias + h) : 0.f, p.delta ? __ldg(p.A + h) : 0.f,
                                value<DT>(p.beta + t * p.beta_s[0] + b * p.beta_s[1] + h));
            s.a[i] = decay_of(gate.log2a);
            s.b[i] = gate.b;
            s.kq[i] = sums[2] * fq * fk;
        }
    }
}

// A block's rows of a state [V,K]: load or zeros, and store.
template <int J>
__device__ __forceinline__ void load_rows(const DeltaParams &p, const float *from, int row0, int l8, float (&s)[kRR][4 * J])
{
#pragma unroll
    for (int r = 0; r < kRR; ++r)
#pragma unroll
        for (int e = 0; e < 4 * J; ++e) {
            const int row = row0 + 4 * r, at = (e / 4) * 32 + l8 * 4 + e % 4;
            s[r][e] = from && row < p.V && at < p.K ? from[row * p.K + at] : 0.f;
        }
}
template <int J>
__device__ __forceinline__ void store_rows(const DeltaParams &p, float *to, int step_row, int step_key, int row0, int l8, const float (&s)[kRR][4 * J])
{
#pragma unroll
    for (int r = 0; r < kRR; ++r)
#pragma unroll
        for (int e = 0; e < 4 * J; ++e) {
            const int row = row0 + 4 * r, at = (e / 4) * 32 + l8 * 4 + e % 4;
            if (row < p.V && at < p.K)
                to[row * step_row + at * step_key] = s[r][e];
        }
}

// This lane's keys of a token.
template <int J>
__device__ __forceinline__ void keys(const float *from, int l8, float (&k)[4 * J])
{
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const float4 v = *reinterpret_cast<const float4 *>(from + j * 32 + l8 * 4);
        k[4 * j] = v.x, k[4 * j + 1] = v.y, k[4 * j + 2] = v.z, k[4 * j + 3] = v.w;
    }
}

template <int N>
__device__ __forceinline__ void sum8(float (&x)[N])
{
#pragma unroll
    for (int d = 1; d < 8; d *= 2)
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] += __shfl_xor_sync(0xFFFFFFFFu, x[i], d);
}

template <int DT, int J>
__global__ void __launch_bounds__(kWarps * 32) mcc1d_delta_tokens_rows(const __grid_constant__ DeltaParams p)
{
    __shared__ TokenShared<32 * J> sh;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l8 = lane % 8;
    const int tiles = (p.V + kRowsPerBlock - 1) / kRowsPerBlock, item = blockIdx.x / tiles;
    const int b = item / p.H, h = item % p.H, first = (blockIdx.x % tiles) * kRowsPerBlock;
    const int mine = warp * 4 * kRR + lane / 8, row0 = first + mine;
    const int64_t n = clamped_length(p.lengths, b, p.S), VK = (int64_t)p.V * p.K;
    float s[kRR][4 * J];
    load_rows<J>(p, p.state ? p.state + item * VK : nullptr, row0, l8, s);
    for (int64_t t0 = 0; t0 < n; t0 += kGroup) {
        const int live = (int)(n - t0 < kGroup ? n - t0 : kGroup);
        if (p.kept.states && t0 % kChunk == 0)
            store_rows<J>(p, p.kept.states + ((t0 / kChunk) * p.B * p.H + item) * p.K * p.kept.Vp, 1, p.kept.Vp, row0, l8, s);
        __syncthreads();
        stage<DT, 32 * J>(p, sh, p.v, p.v_s, b, h, first, t0, live);
        __syncthreads();
        for (int i = 0; i < live; ++i) {
            float k[4 * J], q[4 * J], x[2 * kRR];
            keys<J>(sh.k[i], l8, k);
            keys<J>(sh.q[i], l8, q);
#pragma unroll
            for (int r = 0; r < kRR; ++r) {
                x[r] = x[kRR + r] = 0.f;
#pragma unroll
                for (int e = 0; e < 4 * J; ++e) {
                    x[r] = fmaf(s[r][e], k[e], x[r]);
                    x[kRR + r] = fmaf(s[r][e], q[e], x[kRR + r]);
                }
            }
            sum8(x);
            const float a = sh.a[i], bt = sh.b[i], kq = sh.kq[i];
            const int64_t out = ((t0 + i) * p.B * p.H + item) * p.V;
#pragma unroll
            for (int r = 0; r < kRR; ++r) {
                const float u = bt * fmaf(-a, x[r], sh.w[i][mine + 4 * r]);
#pragma unroll
                for (int e = 0; e < 4 * J; ++e)
                    s[r][e] = fmaf(u, k[e], a * s[r][e]);
                if (l8 == 0 && row0 + 4 * r < p.V) {
                    if (p.y)
                        p.y[out + row0 + 4 * r] = (uint16_t)pack2<DT>(make_float2(fmaf(u, kq, a * x[kRR + r]), 0.f));
                    if (p.kept.u)
                        p.kept.u[((t0 + i) * p.B * p.H + item) * p.kept.Vp + row0 + 4 * r] = u;
                }
            }
        }
    }
    if (p.final_state)
        store_rows<J>(p, p.final_state + item * VK, p.K, 1, row0, l8, s);
    if (p.y)
        for (int64_t t = n + warp; t < p.S; t += kWarps)
            for (int j = lane; j < kRowsPerBlock; j += 32)
                if (first + j < p.V)
                    p.y[(t * p.B * p.H + item) * p.V + first + j] = 0;
}

// The states' gradients backwards. With G the gradient of S(t) from later
// tokens: du = (G + gy q'^T) k', grad_v = b du, and before the token
// G = a (G + gy q'^T - b du k'^T).
template <int DT, int J>
__global__ void __launch_bounds__(kWarps * 32) mcc1d_delta_tokens_bwd_rows(const __grid_constant__ DeltaParams p)
{
    __shared__ TokenShared<32 * J> sh;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l8 = lane % 8;
    const int tiles = (p.V + kRowsPerBlock - 1) / kRowsPerBlock, item = blockIdx.x / tiles;
    const int b = item / p.H, h = item % p.H, first = (blockIdx.x % tiles) * kRowsPerBlock;
    const int mine = warp * 4 * kRR + lane / 8, row0 = first + mine;
    const int64_t n = clamped_length(p.lengths, b, p.S), VK = (int64_t)p.V * p.K;
    float s[kRR][4 * J];
    load_rows<J>(p, p.grad_final ? p.grad_final + item * VK : nullptr, row0, l8, s);
    for (int64_t t0 = (n - 1) / kGroup * kGroup; n > 0 && t0 >= 0; t0 -= kGroup) {
        const int live = (int)(n - t0 < kGroup ? n - t0 : kGroup);
        if ((t0 + kGroup) % kChunk == 0 || t0 + kGroup >= n)
            store_rows<J>(p, p.kept.states + ((t0 / kChunk) * p.B * p.H + item) * p.K * p.kept.Vp, 1, p.kept.Vp, row0, l8, s);
        __syncthreads();
        stage<DT, 32 * J>(p, sh, p.grad_y, p.gy_s, b, h, first, t0, live);
        __syncthreads();
        for (int i = live - 1; i >= 0; --i) {
            float k[4 * J], q[4 * J], x[kRR];
            keys<J>(sh.k[i], l8, k);
            keys<J>(sh.q[i], l8, q);
#pragma unroll
            for (int r = 0; r < kRR; ++r) {
                x[r] = 0.f;
#pragma unroll
                for (int e = 0; e < 4 * J; ++e)
                    x[r] = fmaf(s[r][e], k[e], x[r]);
            }
            sum8(x);
            const float a = sh.a[i], bt = sh.b[i], kq = sh.kq[i];
            const int64_t out = ((t0 + i) * p.B * p.H + item) * p.V;
#pragma unroll
            for (int r = 0; r < kRR; ++r) {
                const float gy = sh.w[i][mine + 4 * r], du = fmaf(gy, kq, x[r]), gm = bt * du;
#pragma unroll
                for (int e = 0; e < 4 * J; ++e)
                    s[r][e] = a * fmaf(-gm, k[e], fmaf(gy, q[e], s[r][e]));
                if (l8 == 0 && row0 + 4 * r < p.V) {
                    p.grad_v[out + row0 + 4 * r] = (uint16_t)pack2<DT>(make_float2(gm, 0.f));
                    p.kept.u[((t0 + i) * p.B * p.H + item) * p.kept.Vp + row0 + 4 * r] = du;
                }
            }
        }
    }
    if (p.grad_state)
        store_rows<J>(p, p.grad_state + item * VK, p.K, 1, row0, l8, s);
    for (int64_t t = n + warp; t < p.S; t += kWarps)
        for (int j = lane; j < kRowsPerBlock; j += 32)
            if (first + j < p.V)
                p.grad_v[(t * p.B * p.H + item) * p.V + first + j] = 0;
}

dim3 token_grid(const DeltaParams &p)
{
    return dim3((unsigned)((int64_t)p.B * p.H * ((p.V + kRowsPerBlock - 1) / kRowsPerBlock)));
}

}  // namespace

int32_t launch_delta_tokens(const mcc1d_delta_args &a, const DeltaKept &kept, cudaStream_t stream)
{
    DeltaParams p = delta_params(a);
    p.kept = kept;
    const auto go = [&](auto kernel) { return launch(kernel, token_grid(p), kWarps * 32, 0, stream, p); };
    if (a.dtype == 0)
        return a.K <= 64 ? go(mcc1d_delta_tokens_rows<0, 2>) : go(mcc1d_delta_tokens_rows<0, 4>);
    return a.K <= 64 ? go(mcc1d_delta_tokens_rows<1, 2>) : go(mcc1d_delta_tokens_rows<1, 4>);
}

int32_t launch_delta_tokens_bwd(const mcc1d_delta_bwd_args &a, const DeltaKept &kept, cudaStream_t stream)
{
    DeltaParams p = delta_params(a.fwd);
    p.kept = kept;
    p.grad_y = static_cast<const uint16_t *>(a.grad_y), p.grad_v = static_cast<uint16_t *>(a.grad_v);
    p.grad_final = a.grad_final_state, p.grad_state = a.grad_state;
    for (int i = 0; i < 3; ++i)
        p.gy_s[i] = a.grad_y_strides[i];
    const auto go = [&](auto kernel) { return launch(kernel, token_grid(p), kWarps * 32, 0, stream, p); };
    if (a.fwd.dtype == 0)
        return a.fwd.K <= 64 ? go(mcc1d_delta_tokens_bwd_rows<0, 2>) : go(mcc1d_delta_tokens_bwd_rows<0, 4>);
    return a.fwd.K <= 64 ? go(mcc1d_delta_tokens_bwd_rows<1, 2>) : go(mcc1d_delta_tokens_bwd_rows<1, 4>);
}

}  // namespace mcc1d
