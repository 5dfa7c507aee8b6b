// delta_step.cu - the gated delta rule of one token per sequence.
//
// The state, 4 V K bytes a head, is read and written once; everything else is
// small beside it. Both products with the state come out of one pass before it
// changes: S(t) q' = a S(t-1) q' + u (k'.q'). States are read and written past the
// caches' order (256 x 16 heads of 128 x 128: 86 us without, 80 with; the copy
// bandwidth would take 79). Loading four values of q and k at once, which leaves
// more blocks in flight, took 93 us.
#include "delta_common.cuh"

namespace mcc1d {

namespace {

struct DeltaStepParams {
    const uint16_t *q, *k, *v, *delta, *beta;
    const float *A, *delta_bias;
    float *state;
    const int32_t *slots;
    uint16_t *y;
    int64_t q_s[2], k_s[2], v_s[2], delta_s, beta_s;
    int64_t cache_rows;
    int32_t H, G, K, V, flags;
    float scale;
    int32_t tiles;       // blocks along V
};

// Eight lanes share a row of the state, each with J groups of four adjacent
// keys 32 apart; a warp has RR times four rows, a block four warps.
constexpr int kStepWarps = 4;

template <int DT, int J, int RR, bool WHOLE>
__global__ void __launch_bounds__(kStepWarps * 32) mcc1d_delta_one_token(const __grid_constant__ DeltaStepParams p)
{
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l8 = lane % 8;
    const uint32_t item = blockIdx.x / p.tiles, tile = blockIdx.x % p.tiles;
    const int b = item / p.H, h = item % p.H, g = h / (p.H / p.G);
    const int row0 = (tile * kStepWarps + warp) * 4 * RR + lane / 8;
    const int64_t slot = p.slots ? (int64_t)__ldg(p.slots + b) : b;
    uint16_t *y = p.y + ((int64_t)b * p.H + h) * p.V;
    if (slot < 0 || slot >= p.cache_rows) {
        if (l8 == 0)
#pragma unroll
            for (int r = 0; r < RR; ++r)
                if (row0 + 4 * r < p.V)
                    y[row0 + 4 * r] = 0;
        return;
    }
    float *state = p.state + ((slot * p.H + h) * p.V) * p.K;
    float4 s[RR][J];
#pragma unroll
    for (int r = 0; r < RR; ++r)
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int row = row0 + 4 * r, at = j * 32 + l8 * 4;
            s[r][j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (WHOLE) {
                if (row < p.V && at < p.K)
                    s[r][j] = __ldcs(reinterpret_cast<const float4 *>(state + row * p.K + at));
            } else if (row < p.V) {
                float *e = reinterpret_cast<float *>(&s[r][j]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at + i < p.K)
                        e[i] = state[row * p.K + at + i];
            }
        }
    const uint16_t *qp = p.q + b * p.q_s[0] + g * p.q_s[1], *kp = p.k + b * p.k_s[0] + g * p.k_s[1];
    float q[4 * J], k[4 * J], sums[3] = {0.f, 0.f, 0.f};       // q.q, k.k, k.q
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int e = 4 * j; e < 4 * j + 4; ++e) {
            const int at = j * 32 + l8 * 4 + e % 4;
            q[e] = at < p.K ? value<DT>(qp + at) : 0.f;
            k[e] = at < p.K ? value<DT>(kp + at) : 0.f;
            sums[0] = fmaf(q[e], q[e], sums[0]);
            sums[1] = fmaf(k[e], k[e], sums[1]);
            sums[2] = fmaf(q[e], k[e], sums[2]);
        }
    }
    const Gates gate = gates_of(p.flags, p.delta != nullptr, p.delta ? value<DT>(p.delta + b * p.delta_s + h) : 0.f,
                                p.delta && p.delta_bias ? __ldg(p.delta_bias + h) : 0.f, p.delta ? __ldg(p.A + h) : 0.f,
                                value<DT>(p.beta + b * p.beta_s + h));
    float pk[RR], pq[RR];
#pragma unroll
    for (int r = 0; r < RR; ++r) {
        pk[r] = pq[r] = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            pk[r] = fmaf(s[r][j].x, k[4 * j], pk[r]), pq[r] = fmaf(s[r][j].x, q[4 * j], pq[r]);
            pk[r] = fmaf(s[r][j].y, k[4 * j + 1], pk[r]), pq[r] = fmaf(s[r][j].y, q[4 * j + 1], pq[r]);
            pk[r] = fmaf(s[r][j].z, k[4 * j + 2], pk[r]), pq[r] = fmaf(s[r][j].z, q[4 * j + 2], pq[r]);
            pk[r] = fmaf(s[r][j].w, k[4 * j + 3], pk[r]), pq[r] = fmaf(s[r][j].w, q[4 * j + 3], pq[r]);
        }
    }
#pragma unroll
    for (int d = 1; d < 8; d *= 2) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            sums[i] += __shfl_xor_sync(0xFFFFFFFFu, sums[i], d);
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            pk[r] += __shfl_xor_sync(0xFFFFFFFFu, pk[r], d);
            pq[r] += __shfl_xor_sync(0xFFFFFFFFu, pq[r], d);
        }
    }
    const float fq = unit_factor(p.flags, sums[0]) * p.scale, fk = unit_factor(p.flags, sums[1]);
    const float a = decay_of(gate.log2a), kq = sums[2] * fq * fk;
#pragma unroll
    for (int r = 0; r < RR; ++r) {
        const int row = row0 + 4 * r;
        if (row >= p.V)
            continue;
        const float v = value<DT>(p.v + b * p.v_s[0] + h * p.v_s[1] + row);
        const float u = gate.b * fmaf(-a * fk, pk[r], v), uk = u * fk;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int at = j * 32 + l8 * 4;
            const float4 o = s[r][j];
            const float4 n = make_float4(fmaf(uk, k[4 * j], a * o.x), fmaf(uk, k[4 * j + 1], a * o.y), fmaf(uk, k[4 * j + 2], a * o.z),
                                         fmaf(uk, k[4 * j + 3], a * o.w));
            if (WHOLE) {
                if (at < p.K)
                    __stcs(reinterpret_cast<float4 *>(state + row * p.K + at), n);
            } else {
                const float e[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at + i < p.K)
                        state[row * p.K + at + i] = e[i];
            }
        }
        if (l8 == 0)
            y[row] = (uint16_t)pack2<DT>(make_float2(fmaf(u, kq, a * fq * pq[r]), 0.f));
    }
}

template <int DT, int J, int RR>
int32_t step(const DeltaStepParams &q, int64_t items, bool whole, cudaStream_t stream)
{
    DeltaStepParams p = q;
    p.tiles = (p.V + 4 * RR * kStepWarps - 1) / (4 * RR * kStepWarps);
    const dim3 grid((unsigned)(items * p.tiles));
    return whole ? launch(mcc1d_delta_one_token<DT, J, RR, true>, grid, kStepWarps * 32, 0, stream, p)
                 : launch(mcc1d_delta_one_token<DT, J, RR, false>, grid, kStepWarps * 32, 0, stream, p);
}

}  // namespace

int32_t launch_delta_step(const mcc1d_delta_step_args &a, cudaStream_t stream)
{
    DeltaStepParams p = {};
    p.q = static_cast<const uint16_t *>(a.q), p.k = static_cast<const uint16_t *>(a.k), p.v = static_cast<const uint16_t *>(a.v);
    p.delta = static_cast<const uint16_t *>(a.delta), p.beta = static_cast<const uint16_t *>(a.beta);
    p.A = a.A, p.delta_bias = a.delta_bias, p.state = a.state, p.slots = a.slots, p.y = static_cast<uint16_t *>(a.y);
    for (int i = 0; i < 2; ++i)
        p.q_s[i] = a.q_strides[i], p.k_s[i] = a.k_strides[i], p.v_s[i] = a.v_strides[i];
    p.delta_s = a.delta_stride, p.beta_s = a.beta_stride, p.cache_rows = a.cache_rows;
    p.H = (int32_t)a.H, p.G = (int32_t)a.G, p.K = (int32_t)a.K, p.V = (int32_t)a.V, p.flags = a.flags, p.scale = (float)a.scale;
    const bool whole = a.K % 4 == 0 && ((uintptr_t)a.state & 15u) == 0;
    const int64_t items = a.B * a.H;
    // Sixteen rows to a warp where that still makes four blocks for each SM: 256
    // sequences of 16 heads of 128 x 128 take 80 us, 84 with eight rows, 93 with
    // four; one sequence takes 2.8 us with four and has an eighth of the blocks
    // with sixteen.
    const bool tall = items * ((a.V + 63) / 64) >= 4 * kNumSMs;
    const auto go = [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        const auto rows = [&](auto rr) {
            constexpr int RR = decltype(rr)::value;
            return a.K <= 32   ? step<DT, 1, RR>(p, items, whole, stream)
                   : a.K <= 64 ? step<DT, 2, RR>(p, items, whole, stream)
                               : step<DT, 4, RR>(p, items, whole, stream);
        };
        return tall ? rows(std::integral_constant<int, 4>()) : rows(std::integral_constant<int, 1>());
    };
    return a.dtype == 0 ? go(std::integral_constant<int, 0>()) : go(std::integral_constant<int, 1>());
}

}  // namespace mcc1d
