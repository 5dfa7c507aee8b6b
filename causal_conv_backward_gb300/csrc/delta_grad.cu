// delta_grad.cu - the gradients of a chunk's q, k, delta and beta, from the
// states before it, the gradients of the state after it, u(t) and du(t).
//
// With c(t) the running sum of log a in the chunk, D(t,i) = exp(c(t) - c(i)) for
// i <= t, S the state before the chunk and G the gradient of the one after it:
//   P'(t,i) = D (gy(t).u(i)),  i <= t;    L'(t,i) = -D (du(t).u(i)),  i < t
//   gq'(t) = e^c(t) gy(t) S + sum over i of P'(t,i) k'(i)
//   gk'(t) = sum over i of P'(i,t) q'(i) + (b(t) L'(t,i) + b(i) L'(i,t)) k'(i)
//            - b(t) e^c(t) du(t) S + e^(c(last) - c(t)) u(t) G
//   gb(t) = du(t).v(t) - e^c(t) (du(t) S).k'(t) + sum over i of L'(t,i) (k'(t).k'(i))
// and what each token's decay multiplies, summed, is the gradient of log a.
#include "delta_common.cuh"

namespace mcc1d {

namespace {

constexpr int kC = kChunk, kVT = 32, kThreads = 256, kPad = kC + 4;

struct GradParams {
    DeltaParams d;
    const float *u, *du, *s, *g;
    uint16_t *grad_q, *grad_k, *grad_delta, *grad_beta;
    float *sum_A, *sum_bias;       // [chunks B][H]
};

template <int KP>
struct GradShared {
    static constexpr int KS = KP + 4;
    float q[kC][KS], k[kC][KS], gq[kC][KS], gk[kC][KS];
    union {
        struct {
            float gy[kVT][kPad], du[kVT][kPad], u[kVT][kPad], s[kVT][KP], g[kVT][KP];
        } in;
        struct {
            float P[kC][kPad], PT[kC][kPad], M[kC][kPad], E[kC][kPad];
        } tri;
    };
    float ch[kC], cl[kC], b[kC], dt[kC], raw[kC], fq[kC], fk[kC], gc[kC], gb[kC], se[kC], dot[8];
};

__device__ __forceinline__ float sum16(float x)
{
#pragma unroll
    for (int d = 1; d < 16; d *= 2)
        x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    return x;
}

template <int DT, int KP>
__global__ void __launch_bounds__(kThreads, 1) delta_grad_kernel(const __grid_constant__ GradParams gp)
{
    extern __shared__ uint8_t raw_shared[];
    typedef GradShared<KP> Shared;
    Shared &sh = *reinterpret_cast<Shared *>(raw_shared);
    constexpr int KC = KP / 16;        // keys of a thread
    const DeltaParams &p = gp.d;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int g = blockIdx.x % p.G, b = (blockIdx.x / p.G) % p.B, per = p.H / p.G;
    const int64_t chunk = blockIdx.x / p.G / p.B, t0 = chunk * kC;
    const int64_t length = clamped_length(p.lengths, b, p.S);
    const int there = (int)(p.S - t0 < kC ? p.S - t0 : kC);                            // rows to write
    const int n = (int)(length <= t0 ? 0 : length - t0 < kC ? length - t0 : kC);       // tokens that are there
    const int64_t BH = (int64_t)p.B * p.H, VK = (int64_t)p.V * p.K;

    // q', k'
    for (int i = warp; i < kC; i += kThreads / 32) {
        const uint16_t *qp = p.q + (t0 + i) * p.q_s[0] + b * p.q_s[1] + g * p.q_s[2];
        const uint16_t *kp = p.k + (t0 + i) * p.k_s[0] + b * p.k_s[1] + g * p.k_s[2];
        float q[KP / 32], k[KP / 32], sums[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
            const int at = j * 32 + lane;
            q[j] = i < n && at < p.K ? value<DT>(qp + at) : 0.f;
            k[j] = i < n && at < p.K ? value<DT>(kp + at) : 0.f;
            sums[0] = fmaf(q[j], q[j], sums[0]);
            sums[1] = fmaf(k[j], k[j], sums[1]);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            sums[0] += __shfl_xor_sync(0xFFFFFFFFu, sums[0], d);
            sums[1] += __shfl_xor_sync(0xFFFFFFFFu, sums[1], d);
        }
        const float fq = unit_factor(p.flags, sums[0]), fk = unit_factor(p.flags, sums[1]);
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
            sh.q[i][j * 32 + lane] = q[j] * (fq * p.scale);
            sh.k[i][j * 32 + lane] = k[j] * fk;
            sh.gq[i][j * 32 + lane] = 0.f;
            sh.gk[i][j * 32 + lane] = 0.f;
        }
        if (lane == 0)
            sh.fq[i] = fq, sh.fk[i] = fk;
    }
    __syncthreads();
    // k'.k' and q'.k' of tokens 4 ty + r and tx + 16 j
    float kk[4][4], qk[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            kk[r][j] = qk[r][j] = 0.f;
    for (int at = 0; at < KP; at += 4) {
        float4 x[4], y[4], z[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            x[r] = *reinterpret_cast<const float4 *>(&sh.k[4 * ty + r][at]);
            y[r] = *reinterpret_cast<const float4 *>(&sh.q[4 * ty + r][at]);
            z[r] = *reinterpret_cast<const float4 *>(&sh.k[tx + 16 * r][at]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                kk[r][j] = fmaf(x[r].x, z[j].x, fmaf(x[r].y, z[j].y, fmaf(x[r].z, z[j].z, fmaf(x[r].w, z[j].w, kk[r][j]))));
                qk[r][j] = fmaf(y[r].x, z[j].x, fmaf(y[r].y, z[j].y, fmaf(y[r].z, z[j].z, fmaf(y[r].w, z[j].w, qk[r][j]))));
            }
    }

    for (int h = g * per; h < (g + 1) * per && n > 0; ++h) {
        const int64_t item = (int64_t)b * p.H + h;
        __syncthreads();
        // gates, and the running sum of log2 a in two parts whose differences are
        // exact in the first: multiples of 2^-9 below 2^14
        if (threadIdx.x < kC) {
            const int i = threadIdx.x;
            const int64_t t = t0 + i;
            Gates gate = {0.f, 0.f, 0.f, 0.f};
            if (i < n)
                gate = gates_of(p.flags, p.delta != nullptr, p.delta ? value<DT>(p.delta + t * p.delta_s[0] + b * p.delta_s[1] + h) : 0.f,
                                p.delta_bias ? __ldg(p.delta_bias + h) : 0.f, p.delta ? __ldg(p.A + h) : 0.f,
                                value<DT>(p.beta + t * p.beta_s[0] + b * p.beta_s[1] + h));
            const float l = fminf(fmaxf(gate.log2a, -255.f), 255.f), hi = rintf(l * 512.f) * (1.f / 512.f);
            sh.ch[i] = hi, sh.cl[i] = l - hi, sh.b[i] = gate.b, sh.dt[i] = gate.dt, sh.raw[i] = gate.raw;
        }
        __syncthreads();
        if (warp < 2) {
            float *c = warp == 0 ? sh.ch : sh.cl;
            float x = c[2 * lane], y = c[2 * lane + 1] + x, s = y;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const float o = __shfl_up_sync(0xFFFFFFFFu, s, d);
                if (lane >= d)
                    s += o;
            }
            const float before = lane > 0 ? __shfl_up_sync(0xFFFFFFFFu, s, 1) : (__shfl_up_sync(0xFFFFFFFFu, s, 1), 0.f);
            c[2 * lane] = before + x;
            c[2 * lane + 1] = before + y;
        }
        __syncthreads();

        float P[4][4], L[4][4], qs[4][KC], ks[4][KC], ke[4][KC], gs = 0.f, dv = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                P[r][j] = L[r][j] = 0.f;
#pragma unroll
            for (int j = 0; j < KC; ++j)
                qs[r][j] = ks[r][j] = ke[r][j] = 0.f;
        }
        const float *S = gp.s + (chunk * BH + item) * VK, *G = gp.g + (chunk * BH + item) * VK;
        for (int v0 = 0; v0 < p.V; v0 += kVT) {
            __syncthreads();
            for (int e = threadIdx.x; e < kC * kVT; e += kThreads) {
                const int i = e / kVT, j = e % kVT;
                const bool live = i < n && v0 + j < p.V;
                const int64_t at = ((t0 + i) * BH + item) * p.V + v0 + j;
                const float du = live ? gp.du[at] : 0.f;
                sh.in.u[j][i] = live ? gp.u[at] : 0.f;
                sh.in.du[j][i] = du;
                sh.in.gy[j][i] = live ? value<DT>(p.grad_y + (t0 + i) * p.gy_s[0] + b * p.gy_s[1] + h * p.gy_s[2] + v0 + j) : 0.f;
            }
            for (int e = threadIdx.x; e < kVT * KP; e += kThreads) {
                const int j = e / KP, at = e % KP;
                const bool live = v0 + j < p.V && at < p.K;
                sh.in.s[j][at] = live ? S[(v0 + j) * p.K + at] : 0.f;
                sh.in.g[j][at] = live ? G[(v0 + j) * p.K + at] : 0.f;
            }
            __syncthreads();
            {   // du.v: four threads to a token
                const int i = threadIdx.x / 4;
                if (i < n)
                    for (int j = threadIdx.x % 4; j < kVT && v0 + j < p.V; j += 4)
                        dv = fmaf(sh.in.du[j][i], value<DT>(p.v + (t0 + i) * p.v_s[0] + b * p.v_s[1] + h * p.v_s[2] + v0 + j), dv);
            }
#pragma unroll 2
            for (int j = 0; j < kVT; ++j) {
                const float4 gy4 = *reinterpret_cast<const float4 *>(&sh.in.gy[j][4 * ty]);
                const float4 du4 = *reinterpret_cast<const float4 *>(&sh.in.du[j][4 * ty]);
                const float4 u4 = *reinterpret_cast<const float4 *>(&sh.in.u[j][4 * ty]);
                const float gy[4] = {gy4.x, gy4.y, gy4.z, gy4.w}, du[4] = {du4.x, du4.y, du4.z, du4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
                float uc[4], s[KC], w[KC];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    uc[c] = sh.in.u[j][tx + 16 * c];
#pragma unroll
                for (int c = 0; c < KC; c += 4) {
                    const float4 s4 = *reinterpret_cast<const float4 *>(&sh.in.s[j][(c / 4) * 64 + 4 * tx]);
                    const float4 g4 = *reinterpret_cast<const float4 *>(&sh.in.g[j][(c / 4) * 64 + 4 * tx]);
                    s[c] = s4.x, s[c + 1] = s4.y, s[c + 2] = s4.z, s[c + 3] = s4.w;
                    w[c] = g4.x, w[c + 1] = g4.y, w[c + 2] = g4.z, w[c + 3] = g4.w;
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        P[r][c] = fmaf(gy[r], uc[c], P[r][c]);
                        L[r][c] = fmaf(-du[r], uc[c], L[r][c]);
                    }
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        qs[r][c] = fmaf(gy[r], s[c], qs[r][c]);
                        ks[r][c] = fmaf(du[r], s[c], ks[r][c]);
                        ke[r][c] = fmaf(u[r], w[c], ke[r][c]);
                    }
                }
                if (j % 16 == ty)
#pragma unroll
                    for (int c = 0; c < KC; ++c)
                        gs = fmaf(s[c], w[c], gs);
            }
        }
        __syncthreads();
        // sum of G S over the block, du.v
#pragma unroll
        for (int d = 16; d > 0; d /= 2)
            gs += __shfl_xor_sync(0xFFFFFFFFu, gs, d);
        if (lane == 0)
            sh.dot[warp] = gs;
        dv += __shfl_xor_sync(0xFFFFFFFFu, dv, 1);
        dv += __shfl_xor_sync(0xFFFFFFFFu, dv, 2);
        if (threadIdx.x % 4 == 0)
            sh.gb[threadIdx.x / 4] = dv;
        const float last_h = sh.ch[kC - 1], last_l = sh.cl[kC - 1];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * ty + r;
            const float th = sh.ch[t], tl = sh.cl[t], bt = sh.b[t];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int i = tx + 16 * c;
                const float D = i <= t ? ex2(fminf((th - sh.ch[i]) + (tl - sh.cl[i]), 127.f)) : 0.f;
                const float pd = P[r][c] * D, ld = i < t ? L[r][c] * D : 0.f;
                sh.tri.E[t][i] = fmaf(pd, qk[r][c], bt * ld * kk[r][c]);
                sh.tri.P[t][i] = pd;
                sh.tri.PT[i][t] = pd;
                L[r][c] = ld;
            }
        }
        float row[4];     // of L' kk
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            row[r] = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                row[r] = fmaf(L[r][c], kk[r][c], row[r]);
            row[r] = sum16(row[r]);
        }
        // M = b L' and its mirror image
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int t = 4 * ty + r, i = tx + 16 * c;
                if (i <= t)
                    sh.tri.M[t][i] = sh.tri.M[i][t] = L[r][c] * sh.b[t];
            }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * ty + r;
            const float ec = ex2(fminf(sh.ch[t] + sh.cl[t], 127.f)), el = ex2(fminf((last_h - sh.ch[t]) + (last_l - sh.cl[t]), 127.f));
            float sq = 0.f, sk = 0.f, se = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int at = (c / 4) * 64 + 4 * tx + c % 4;
                const float q = sh.q[t][at], k = sh.k[t][at];
                qs[r][c] *= ec, ks[r][c] *= -ec, ke[r][c] *= el;
                sq = fmaf(qs[r][c], q, sq);
                sk = fmaf(ks[r][c], k, sk);
                se = fmaf(ke[r][c], k, se);
                ke[r][c] = fmaf(ks[r][c], sh.b[t], ke[r][c]);
            }
            sq = sum16(sq), sk = sum16(sk), se = sum16(se);
            if (tx == 0) {
                sh.gc[t] = sq + sh.b[t] * sk - se;
                sh.se[t] = se;
                sh.gb[t] += sk + row[r];
            }
        }
        __syncthreads();
        // the token's own products
        for (int i = 0; i < kC; ++i) {
            const float4 p4 = *reinterpret_cast<const float4 *>(&sh.tri.PT[i][4 * ty]), pt4 = *reinterpret_cast<const float4 *>(&sh.tri.P[i][4 * ty]);
            const float4 m4 = *reinterpret_cast<const float4 *>(&sh.tri.M[i][4 * ty]);
            const float pr[4] = {p4.x, p4.y, p4.z, p4.w}, pt[4] = {pt4.x, pt4.y, pt4.z, pt4.w}, m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int at = (c / 4) * 64 + 4 * tx + c % 4;
                const float q = sh.q[i][at], k = sh.k[i][at];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    qs[r][c] = fmaf(pr[r], k, qs[r][c]);
                    ke[r][c] = fmaf(pt[r], q, fmaf(m[r], k, ke[r][c]));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const int at = (c / 4) * 64 + 4 * tx + c % 4;
                sh.gq[4 * ty + r][at] += qs[r][c];
                sh.gk[4 * ty + r][at] += ke[r][c];
            }
        if (threadIdx.x < kC) {
            const int t = threadIdx.x;
            float x = sh.gc[t];
            for (int i = 0; i < kC; ++i)
                x += sh.tri.E[t][i] - sh.tri.E[i][t];
            if (t == kC - 1) {
                float s = 0.f;
                for (int w = 0; w < kThreads / 32; ++w)
                    s += sh.dot[w];
                s *= ex2(fminf(last_h + last_l, 127.f));
                for (int i = 0; i < kC; ++i)
                    s += sh.se[i];
                x += s;
            }
            sh.gc[t] = x;
        }
        __syncthreads();
        if (warp == 0) {
            float x = sh.gc[2 * lane + 1], y = sh.gc[2 * lane] + x, s = y;      // sums to the end
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const float o = __shfl_down_sync(0xFFFFFFFFu, s, d);
                if (lane + d < 32)
                    s += o;
            }
            const float o = __shfl_down_sync(0xFFFFFFFFu, s, 1), after = lane < 31 ? o : 0.f;
            const float A = p.delta ? __ldg(p.A + h) : 0.f;
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                const float gl = i < n ? after + (e ? x : y) : 0.f;
                float graw = gl * A;
                if (p.flags & MCC1D_SOFTPLUS)
                    graw *= sigmoid(sh.raw[i]);
                float gbeta = i < n ? sh.gb[i] : 0.f;
                if (p.flags & MCC1D_SIGMOID)
                    gbeta *= sh.b[i] * (1.f - sh.b[i]);
                if (i < there) {
                    const int64_t at = ((t0 + i) * p.B + b) * p.H + h;
                    gp.grad_beta[at] = (uint16_t)pack2<DT>(make_float2(gbeta, 0.f));
                    if (gp.grad_delta)
                        gp.grad_delta[at] = (uint16_t)pack2<DT>(make_float2(graw, 0.f));
                }
                sa = fmaf(gl, sh.dt[i], sa);
                sb += graw;
            }
#pragma unroll
            for (int d = 16; d > 0; d /= 2) {
                sa += __shfl_xor_sync(0xFFFFFFFFu, sa, d);
                sb += __shfl_xor_sync(0xFFFFFFFFu, sb, d);
            }
            if (lane == 0) {
                gp.sum_A[(chunk * p.B + b) * p.H + h] = sa;
                gp.sum_bias[(chunk * p.B + b) * p.H + h] = sb;
            }
        }
    }
    __syncthreads();
    if (n == 0)
        for (int e = threadIdx.x; e < kC * per; e += kThreads) {
            const int i = e / per, h = g * per + e % per;
            if (i < there) {
                const int64_t at = ((t0 + i) * p.B + b) * p.H + h;
                gp.grad_beta[at] = 0;
                if (gp.grad_delta)
                    gp.grad_delta[at] = 0;
            }
            if (i == 0)
                gp.sum_A[(chunk * p.B + b) * p.H + h] = gp.sum_bias[(chunk * p.B + b) * p.H + h] = 0.f;
        }
    // through the division by the lengths: (g - x (x.g)) f for a unit vector x
    const float inverse = p.scale != 0.f ? 1.f / (p.scale * p.scale) : 0.f;
    for (int i = warp; i < there; i += kThreads / 32) {
        const bool norm = p.flags & MCC1D_QK_NORM;
        float dq = 0.f, dk = 0.f;
        for (int at = lane; at < KP; at += 32) {
            dq = fmaf(sh.gq[i][at], sh.q[i][at], dq);
            dk = fmaf(sh.gk[i][at], sh.k[i][at], dk);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            dq += __shfl_xor_sync(0xFFFFFFFFu, dq, d);
            dk += __shfl_xor_sync(0xFFFFFFFFu, dk, d);
        }
        dq = norm ? dq * inverse : 0.f, dk = norm ? dk : 0.f;
        const float fq = sh.fq[i] * p.scale, fk = sh.fk[i];
        const int64_t to = (((t0 + i) * p.B + b) * p.G + g) * p.K;
        for (int at = lane; at < p.K; at += 32) {
            gp.grad_q[to + at] = (uint16_t)pack2<DT>(make_float2(fmaf(-sh.q[i][at], dq, sh.gq[i][at]) * fq, 0.f));
            gp.grad_k[to + at] = (uint16_t)pack2<DT>(make_float2(fmaf(-sh.k[i][at], dk, sh.gk[i][at]) * fk, 0.f));
        }
    }
}

template <int DT, int KP>
int32_t grad(const GradParams &p, int64_t blocks, cudaStream_t stream)
{
    constexpr int bytes = (int)sizeof(GradShared<KP>);
    if (cudaFuncSetAttribute(delta_grad_kernel<DT, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return kErrCuda;
    return launch(delta_grad_kernel<DT, KP>, dim3((unsigned)blocks), kThreads, bytes, stream, p);
}

}  // namespace

DeltaBwdPlan delta_bwd_plan(const mcc1d_delta_bwd_args &a)
{
    const mcc1d_delta_args &f = a.fwd;
    DeltaBwdPlan p = {};
    p.chunks = (f.S + kChunk - 1) / kChunk;
    const auto take = [&](int64_t floats) {
        const uint64_t at = p.bytes;
        p.bytes += ((uint64_t)floats * 4 + 255) / 256 * 256;
        return at;
    };
    const int64_t tokens = f.S * f.B * f.H * f.V, states = p.chunks * f.B * f.H * f.V * f.K;
    p.off_u = take(tokens), p.off_du = take(tokens);
    p.off_s = take(states), p.off_g = take(states);
    p.off_sums = take(2 * p.chunks * f.B * f.H);
    return p;
}

int32_t launch_delta_bwd(const mcc1d_delta_bwd_args &a, void *workspace, cudaStream_t stream)
{
    const mcc1d_delta_args &f = a.fwd;
    const DeltaBwdPlan plan = delta_bwd_plan(a);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const auto at = [&](uint64_t off) { return reinterpret_cast<float *>(ws + off); };
    mcc1d_delta_args in = f;
    in.y = nullptr, in.final_state = nullptr;
    int32_t st = launch_delta_tokens(in, at(plan.off_u), at(plan.off_s), stream);
    if (st == kOk)
        st = launch_delta_tokens_bwd(a, at(plan.off_du), at(plan.off_g), stream);
    if (st != kOk)
        return st;
    GradParams p = {};
    p.d = delta_params(in);
    p.d.grad_y = static_cast<const uint16_t *>(a.grad_y);
    for (int i = 0; i < 3; ++i)
        p.d.gy_s[i] = a.grad_y_strides[i];
    p.u = at(plan.off_u), p.du = at(plan.off_du), p.s = at(plan.off_s), p.g = at(plan.off_g);
    p.grad_q = static_cast<uint16_t *>(a.grad_q), p.grad_k = static_cast<uint16_t *>(a.grad_k);
    p.grad_delta = f.delta ? static_cast<uint16_t *>(a.grad_delta) : nullptr, p.grad_beta = static_cast<uint16_t *>(a.grad_beta);
    const int64_t parts = plan.chunks * f.B;
    p.sum_A = at(plan.off_sums), p.sum_bias = p.sum_A + parts * f.H;
    const int64_t blocks = parts * f.G;
    if (f.dtype == 0)
        st = f.K <= 64 ? grad<0, 64>(p, blocks, stream) : grad<0, 128>(p, blocks, stream);
    else
        st = f.K <= 64 ? grad<1, 64>(p, blocks, stream) : grad<1, 128>(p, blocks, stream);
    if (st != kOk || !f.delta)
        return st;
    const ColumnSums s = {{p.sum_A, p.sum_bias}, {a.grad_A, f.delta_bias ? a.grad_delta_bias : nullptr}, {2, 2}};
    return launch_column_sums(s, parts, f.H, 2, stream);
}

}  // namespace mcc1d
