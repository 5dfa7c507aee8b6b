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
//
// All products are on the tensor cores with fp32 operands as two tf32 terms
// (22 bits, any range; grad_y, q and k are exact in one), by mma.sync: the sums
// behind grad_A and grad_delta_bias run over all tokens, and would show less.
// They bound the kernel: 84 per eight values of V, 48 per eight tokens, a warp.
#include "delta_common.cuh"

namespace mcc1d {

namespace {

constexpr int kC = kChunk, kVT = 32, kThreads = 256, kTri = kC + 4, kVS = kVT + 4, kRaw = kVT + 8;

struct GradParams {
    DeltaParams d;
    const float *u, *du, *s, *g;   // [S,B,H,Vp], [chunks][B H][K,Vp]
    int32_t Vp;
    bool vectors_gy, vectors_v;
    uint16_t *grad_q, *grad_k, *grad_delta, *grad_beta;
    float *sum_A, *sum_bias;       // [chunks B][H]
};

// Strides are 4 or 8 over a multiple of 32 words, so that the eight rows and
// four columns (or the other way round) of a fragment lie on different banks.
template <int KP>
struct GradTile {
    float u[kC][kVS], du[kC][kVS], s[KP][kVS], g[KP][kVS];
    uint16_t gy[kC][kRaw], v[kC][kRaw];
};
template <int KP>
struct GradShared {
    static constexpr int KS = KP + 8;
    float q[kC][KS], k[kC][KS];        // as they are, not divided by their lengths
    union {
        GradTile<KP> tile[2];
        struct {
            float P[kC][kTri], PT[kC][kTri], M[kC][kTri];
        };
    };
    float ch[kC], cl[kC], b[kC], dt[kC], raw[kC], fq[kC], fk[kC], gc[kC], gb[kC], dv[kC], dot[8];
    float sq[2][kC], sk[2][kC], se[2][kC], row[2][kC], low[2][kC], col[4][kC];     // of the warps that share a row or column
};

// A value as two tf32 terms, 22 bits.
struct Terms {
    uint32_t hi, lo;
};
__device__ __forceinline__ uint32_t tf32(float x)
{
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ Terms terms(float x)
{
    Terms t;
    t.hi = tf32(x);
    t.lo = tf32(x - __uint_as_float(t.hi));
    return t;
}
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += (a) (b), a exact or of two terms, the small products first
__device__ __forceinline__ void mma_exact_a(float (&c)[4], const uint32_t (&a)[4], const Terms &b0, const Terms &b1)
{
    mma1688(c, a, b0.lo, b1.lo);
    mma1688(c, a, b0.hi, b1.hi);
}
// The tensor cores cut their sums off where fp32 would round: long sums are
// taken eight products at a time and added outside.
__device__ __forceinline__ void add4(float (&c)[4], const float (&x)[4])
{
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const float2 s = add2(make_float2(c[e], c[e + 1]), make_float2(x[e], x[e + 1]));
        c[e] = s.x, c[e + 1] = s.y;
    }
}
__device__ __forceinline__ void mma_terms(float (&c)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4], const Terms &b0, const Terms &b1)
{
    mma1688(c, hi, b0.lo, b1.lo);
    mma1688(c, lo, b0.hi, b1.hi);
    mma1688(c, hi, b0.hi, b1.hi);
}
// The 16 x 8 fragment at rows r.., columns c.. of a row-major matrix.
template <int STRIDE>
__device__ __forceinline__ void fragment(const float (*m)[STRIDE], int r, int c, uint32_t (&hi)[4], uint32_t (&lo)[4])
{
    const int g = threadIdx.x % 32 / 4, t = threadIdx.x % 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const Terms x = terms(m[r + g + 8 * (e % 2)][c + t + 4 * (e / 2)]);
        hi[e] = x.hi, lo[e] = x.lo;
    }
}

__device__ __forceinline__ float sum4(float x)
{
    x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
    return x + __shfl_xor_sync(0xFFFFFFFFu, x, 2);
}

__device__ __forceinline__ void copy16(void *to, const void *from, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(bytes) : "memory");
}

// Values v0.. of a chunk's rows: u, du, grad_y, v, and of the states' rows.
template <int DT, int KP>
__device__ __forceinline__ void bring(const GradParams &gp, GradTile<KP> &tile, int64_t chunk, int64_t item, int b, int h, int n, int v0)
{
    const DeltaParams &p = gp.d;
    const int64_t BH = (int64_t)p.B * p.H, t0 = chunk * kC;
    const int tid = threadIdx.x;
#pragma unroll 2
    for (int e = tid; e < kC * kVT / 4; e += kThreads) {
        const int t = e / (kVT / 4), at = 4 * (e % (kVT / 4));
        const bool live = t < n && v0 + at < gp.Vp;
        const int64_t from = live ? ((t0 + t) * BH + item) * gp.Vp + v0 + at : 0;
        const int bytes = live ? max(0, min(4, p.V - v0 - at)) * 4 : 0;
        copy16(&tile.u[t][at], gp.u + from, bytes);
        copy16(&tile.du[t][at], gp.du + from, bytes);
    }
    const int64_t first = (chunk * BH + item) * p.K * gp.Vp + v0;
#pragma unroll 2
    for (int e = tid; e < KP * kVT / 4; e += kThreads) {
        const int k = e / (kVT / 4), at = 4 * (e % (kVT / 4));
        const bool live = k < p.K && v0 + at < gp.Vp;
        const int64_t from = live ? first + (int64_t)k * gp.Vp + at : 0;
        const int bytes = live ? max(0, min(4, p.V - v0 - at)) * 4 : 0;
        copy16(&tile.s[k][at], gp.s + from, bytes);
        copy16(&tile.g[k][at], gp.g + from, bytes);
    }
    // 16-bit rows: eight values to a thread, 64 rows
    const int t = tid / 4, at = 8 * (tid % 4), live = t < n ? p.V - v0 - at : 0;
    const uint16_t *gy = p.grad_y + (t0 + t) * p.gy_s[0] + b * p.gy_s[1] + h * p.gy_s[2] + v0 + at;
    const uint16_t *v = p.v + (t0 + t) * p.v_s[0] + b * p.v_s[1] + h * p.v_s[2] + v0 + at;
    if (gp.vectors_gy)
        copy16(&tile.gy[t][at], live > 0 ? gy : p.grad_y, live > 0 ? 16 : 0);
    else
        for (int i = 0; i < 8; ++i)
            tile.gy[t][at + i] = i < live ? __ldg(gy + i) : (uint16_t)0;
    if (gp.vectors_v)
        copy16(&tile.v[t][at], live > 0 ? v : p.v, live > 0 ? 16 : 0);
    else
        for (int i = 0; i < 8; ++i)
            tile.v[t][at + i] = i < live ? __ldg(v + i) : (uint16_t)0;
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int DT, int KP>
__global__ void __launch_bounds__(kThreads, 1) delta_grad_kernel(const __grid_constant__ GradParams gp)
{
    extern __shared__ __align__(16) uint8_t raw_shared[];
    typedef GradShared<KP> Shared;
    Shared &sh = *reinterpret_cast<Shared *>(raw_shared);
    constexpr int NK = KP / 16;        // eights of keys of a warp
    const DeltaParams &p = gp.d;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, fg = lane / 4, ft = lane % 4;
    // a warp has 16 tokens, half of the other tokens and half of the keys
    const int r0 = 16 * (warp % 4), part = warp / 4, c0 = 32 * part, k0 = KP / 2 * part;
    const int g = blockIdx.x % p.G, b = (blockIdx.x / p.G) % p.B, per = p.H / p.G;
    const int64_t chunk = blockIdx.x / p.G / p.B, t0 = chunk * kC;
    const int64_t length = clamped_length(p.lengths, b, p.S);
    const int there = (int)(p.S - t0 < kC ? p.S - t0 : kC);                            // rows to write
    const int n = (int)(length <= t0 ? 0 : length - t0 < kC ? length - t0 : kC);       // tokens that are there
    const int tiles = (p.V + kVT - 1) / kVT;

    // q, k and what they are multiplied by
    for (int i = warp; i < kC; i += kThreads / 32) {
        const uint16_t *qp = p.q + (t0 + i) * p.q_s[0] + b * p.q_s[1] + g * p.q_s[2];
        const uint16_t *kp = p.k + (t0 + i) * p.k_s[0] + b * p.k_s[1] + g * p.k_s[2];
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
            const int at = j * 32 + lane;
            const float q = i < n && at < p.K ? value<DT>(qp + at) : 0.f, k = i < n && at < p.K ? value<DT>(kp + at) : 0.f;
            sums[0] = fmaf(q, q, sums[0]);
            sums[1] = fmaf(k, k, sums[1]);
            sh.q[i][at] = q, sh.k[i][at] = k;
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            sums[0] += __shfl_xor_sync(0xFFFFFFFFu, sums[0], d);
            sums[1] += __shfl_xor_sync(0xFFFFFFFFu, sums[1], d);
        }
        if (lane == 0)
            sh.fq[i] = unit_factor(p.flags, sums[0]), sh.fk[i] = unit_factor(p.flags, sums[1]);
    }
    float gq[NK][4], gk[NK][4];        // of q', k', over the heads that share them
#pragma unroll
    for (int j = 0; j < NK; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            gq[j][e] = gk[j][e] = 0.f;

    for (int h = g * per; h < (g + 1) * per && n > 0; ++h) {
        const int64_t item = (int64_t)b * p.H + h;
        __syncthreads();
        bring<DT, KP>(gp, sh.tile[0], chunk, item, b, h, n, 0);
        // gates, and the running sum of log2 a in two parts whose differences are
        // exact in the first: multiples of 2^-9 below 2^14
        if (tid < kC) {
            const int64_t t = t0 + tid;
            Gates gate = {0.f, 0.f, 0.f, 0.f};
            if (tid < n)
                gate = gates_of(p.flags, p.delta != nullptr, p.delta ? value<DT>(p.delta + t * p.delta_s[0] + b * p.delta_s[1] + h) : 0.f,
                                p.delta_bias ? __ldg(p.delta_bias + h) : 0.f, p.delta ? __ldg(p.A + h) : 0.f,
                                value<DT>(p.beta + t * p.beta_s[0] + b * p.beta_s[1] + h));
            const float l = fminf(fmaxf(gate.log2a, -255.f), 255.f), hi = rintf(l * 512.f) * (1.f / 512.f);
            sh.ch[tid] = hi, sh.cl[tid] = l - hi, sh.b[tid] = gate.b, sh.dt[tid] = gate.dt, sh.raw[tid] = gate.raw;
        }
        __syncthreads();
        if (warp < 2) {
            float *c = warp == 0 ? sh.ch : sh.cl;
            const float x = c[2 * lane], y = c[2 * lane + 1] + x;
            float s = y;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const float o = __shfl_up_sync(0xFFFFFFFFu, s, d);
                if (lane >= d)
                    s += o;
            }
            const float o = __shfl_up_sync(0xFFFFFFFFu, s, 1), before = lane > 0 ? o : 0.f;
            c[2 * lane] = before + x;
            c[2 * lane + 1] = before + y;
        }

        float P[4][4] = {}, L[4][4] = {}, qs[NK][4] = {}, ks[NK][4] = {}, ke[NK][4] = {}, gs = 0.f, dv = 0.f;
        const bool low = c0 <= r0 + 15;        // some of the other tokens are not after the warp's
        for (int tile = 0; tile < tiles; ++tile) {
            if (tile + 1 < tiles) {
                bring<DT, KP>(gp, sh.tile[(tile + 1) % 2], chunk, item, b, h, n, (tile + 1) * kVT);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncthreads();
            const GradTile<KP> &x = sh.tile[tile % 2];
#pragma unroll 1
            for (int v = 0; v < kVT; v += 8) {
                uint32_t gy[4], duh[4], dul[4], uh[4], ul[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    gy[e] = __float_as_uint(unpack2<DT>(x.gy[r0 + fg + 8 * (e % 2)][v + ft + 4 * (e / 2)]).x);
                fragment<kVS>(x.du, r0, v, duh, dul);
                fragment<kVS>(x.u, r0, v, uh, ul);
                if (low)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const Terms u0 = terms(x.u[c0 + 8 * j + fg][v + ft]), u1 = terms(x.u[c0 + 8 * j + fg][v + ft + 4]);
                        float x[4] = {}, y[4] = {};
                        mma_exact_a(x, gy, u0, u1);
                        mma_terms(y, duh, dul, u0, u1);
                        add4(P[j], x), add4(L[j], y);
                    }
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    const int at = k0 + 8 * j + fg;
                    const Terms s0 = terms(x.s[at][v + ft]), s1 = terms(x.s[at][v + ft + 4]);
                    float x4[4] = {}, y4[4] = {}, z4[4] = {};
                    mma_exact_a(x4, gy, s0, s1);
                    mma_terms(y4, duh, dul, s0, s1);
                    const Terms g0 = terms(x.g[at][v + ft]), g1 = terms(x.g[at][v + ft + 4]);
                    mma_terms(z4, uh, ul, g0, g1);
                    add4(qs[j], x4), add4(ks[j], y4), add4(ke[j], z4);
                }
            }
            for (int e = tid; e < kVT * KP; e += kThreads)
                gs = fmaf(x.s[e / kVT][e % kVT], x.g[e / kVT][e % kVT], gs);
#pragma unroll
            for (int j = 0; j < 8; ++j)           // du.v: four threads to a token
                dv = fmaf(x.du[tid / 4][8 * (tid % 4) + j], unpack2<DT>(x.v[tid / 4][8 * (tid % 4) + j]).x, dv);
            __syncthreads();
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2)
            gs += __shfl_xor_sync(0xFFFFFFFFu, gs, d);
        if (lane == 0)
            sh.dot[warp] = gs;
        dv = sum4(dv);
        if (tid % 4 == 0)
            sh.dv[tid / 4] = dv;
        const float last_h = sh.ch[kC - 1], last_l = sh.cl[kC - 1];
        // the states' parts, and what they say about the decays
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = r0 + fg + 8 * half;
            const float ec = ex2(fminf(sh.ch[t] + sh.cl[t], 127.f)), el = ex2(fminf((last_h - sh.ch[t]) + (last_l - sh.cl[t]), 127.f));
            const float bt = sh.b[t];
            float sq = 0.f, sk = 0.f, se = 0.f;
#pragma unroll
            for (int j = 0; j < NK; ++j)
#pragma unroll
                for (int e = 2 * half; e < 2 * half + 2; ++e) {
                    const int at = k0 + 8 * j + 2 * ft + e % 2;
                    const float q = sh.q[t][at], k = sh.k[t][at], x = ec * qs[j][e], y = -ec * ks[j][e], z = el * ke[j][e];
                    sq = fmaf(x, q, sq);
                    sk = fmaf(y, k, sk);
                    se = fmaf(z, k, se);
                    gq[j][e] += x;
                    gk[j][e] += fmaf(bt, y, z);
                }
            sq = sum4(sq), sk = sum4(sk), se = sum4(se);
            if (ft == 0) {
                sh.sq[part][t] = sq * (sh.fq[t] * p.scale);
                sh.sk[part][t] = sk * sh.fk[t];
                sh.se[part][t] = se * sh.fk[t];
            }
        }
        {   // k.k, q.k in the place of the states' parts: exact in one term each
            float kk[4][4] = {}, qk[4][4] = {};
            if (low)
#pragma unroll 2
                for (int at = 0; at < KP; at += 8) {
                    uint32_t aq[4], ak[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        aq[e] = __float_as_uint(sh.q[r0 + fg + 8 * (e % 2)][at + ft + 4 * (e / 2)]);
                        ak[e] = __float_as_uint(sh.k[r0 + fg + 8 * (e % 2)][at + ft + 4 * (e / 2)]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t x = __float_as_uint(sh.k[c0 + 8 * j + fg][at + ft]), y = __float_as_uint(sh.k[c0 + 8 * j + fg][at + ft + 4]);
                        mma1688(kk[j], ak, x, y);
                        mma1688(qk[j], aq, x, y);
                    }
                }
            float col[4][2] = {};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int t = r0 + fg + 8 * half;
                const float th = sh.ch[t], tl = sh.cl[t], bt = sh.b[t], fkt = sh.fk[t], fqt = sh.fq[t] * p.scale;
                float row = 0.f, lowrow = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int i = c0 + 8 * j + 2 * ft + e, x = 2 * half + e;
                        const float fki = sh.fk[i];
                        const float D = i <= t ? ex2(fminf((th - sh.ch[i]) + (tl - sh.cl[i]), 127.f)) : 0.f;
                        const float pd = i <= t ? P[j][x] * D : 0.f, ld = i < t ? -L[j][x] * D : 0.f, lk = ld * (kk[j][x] * fkt * fki);
                        const float E = fmaf(pd, qk[j][x] * fqt * fki, bt * lk);
                        row += E, lowrow += lk, col[j][e] += E;
                        sh.P[t][i] = pd * fki;
                        sh.PT[i][t] = pd * fqt;
                        if (i <= t) {
                            sh.M[t][i] = bt * ld * fki;
                            sh.M[i][t] = bt * ld * fkt;
                        }
                    }
                row = sum4(row), lowrow = sum4(lowrow);
                if (ft == 0)
                    sh.row[part][t] = row, sh.low[part][t] = lowrow;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float c = col[j][e];
#pragma unroll
                    for (int d = 4; d < 32; d *= 2)
                        c += __shfl_xor_sync(0xFFFFFFFFu, c, d);
                    if (fg == 0)
                        sh.col[warp % 4][c0 + 8 * j + 2 * ft + e] = c;
                }
        }
        __syncthreads();
        // the tokens' own products, of two terms and q or k as they are
#pragma unroll 1
        for (int i = 0; i < kC; i += 8) {
            uint32_t ph[4], pl[4], th[4], tl[4], mh[4], ml[4];
            fragment<kTri>(sh.P, r0, i, ph, pl);
            fragment<kTri>(sh.PT, r0, i, th, tl);
            fragment<kTri>(sh.M, r0, i, mh, ml);
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                const int at = k0 + 8 * j + fg;
                const uint32_t q0 = __float_as_uint(sh.q[i + ft][at]), q1 = __float_as_uint(sh.q[i + ft + 4][at]);
                const uint32_t x0 = __float_as_uint(sh.k[i + ft][at]), x1 = __float_as_uint(sh.k[i + ft + 4][at]);
                mma1688(gq[j], ph, x0, x1);
                mma1688(gq[j], pl, x0, x1);
                mma1688(gk[j], th, q0, q1);
                mma1688(gk[j], tl, q0, q1);
                mma1688(gk[j], mh, x0, x1);
                mma1688(gk[j], ml, x0, x1);
            }
        }
        if (warp == 0) {
            const float A = p.delta ? __ldg(p.A + h) : 0.f;
            float x[2], all_e = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                const float se = sh.se[0][t] + sh.se[1][t], sk = sh.sk[0][t] + sh.sk[1][t];
                x[e] = (sh.row[0][t] + sh.row[1][t]) - ((sh.col[0][t] + sh.col[1][t]) + (sh.col[2][t] + sh.col[3][t]));
                x[e] += (sh.sq[0][t] + sh.sq[1][t]) + sh.b[t] * sk - se;
                sh.gb[t] = sh.dv[t] + sk + (sh.low[0][t] + sh.low[1][t]);
                all_e += se;
            }
#pragma unroll
            for (int d = 16; d > 0; d /= 2)
                all_e += __shfl_xor_sync(0xFFFFFFFFu, all_e, d);
            if (lane == 31) {
                float s = 0.f;
                for (int w = 0; w < kThreads / 32; ++w)
                    s += sh.dot[w];
                x[1] += fmaf(s, ex2(fminf(last_h + last_l, 127.f)), all_e);
            }
            const float y = x[0] + x[1];
            float s = y;      // sums to the end
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const float o = __shfl_down_sync(0xFFFFFFFFu, s, d);
                if (lane + d < 32)
                    s += o;
            }
            const float o = __shfl_down_sync(0xFFFFFFFFu, s, 1), after = lane < 31 ? o : 0.f;
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                const float gl = i < n ? after + (e ? x[1] : y) : 0.f;
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
        for (int e = tid; e < kC * per; e += kThreads) {
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
    const bool norm = p.flags & MCC1D_QK_NORM;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int t = r0 + fg + 8 * half;
        float dq = 0.f, dk = 0.f;
#pragma unroll
        for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int at = k0 + 8 * j + 2 * ft + e;
                dq = fmaf(gq[j][2 * half + e], sh.q[t][at], dq);
                dk = fmaf(gk[j][2 * half + e], sh.k[t][at], dk);
            }
        dq = sum4(dq), dk = sum4(dk);
        if (ft == 0)
            sh.sq[part][t] = dq, sh.sk[part][t] = dk;
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int t = r0 + fg + 8 * half;
        if (t >= there)
            continue;
        const float fq = sh.fq[t], fk = sh.fk[t];
        const float dq = norm ? (sh.sq[0][t] + sh.sq[1][t]) * fq * fq : 0.f, dk = norm ? (sh.sk[0][t] + sh.sk[1][t]) * fk * fk : 0.f;
        const int64_t to = (((t0 + t) * p.B + b) * p.G + g) * p.K;
#pragma unroll
        for (int j = 0; j < NK; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int at = k0 + 8 * j + 2 * ft + e;
                if (at < p.K) {
                    gp.grad_q[to + at] = (uint16_t)pack2<DT>(make_float2(fmaf(-sh.q[t][at], dq, gq[j][2 * half + e]) * (fq * p.scale), 0.f));
                    gp.grad_k[to + at] = (uint16_t)pack2<DT>(make_float2(fmaf(-sh.k[t][at], dk, gk[j][2 * half + e]) * fk, 0.f));
                }
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
    p.Vp = (int32_t)((f.V + 3) / 4 * 4);
    p.tokens = delta_plan(f).tokens;
    const auto take = [&](uint64_t bytes) {
        const uint64_t at = p.bytes;
        p.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    const uint64_t tokens = (uint64_t)(f.S * f.B * f.H) * p.Vp, states = (uint64_t)(p.chunks * f.B * f.H * f.K) * p.Vp;
    p.off_u = take(4 * tokens), p.off_du = take(4 * tokens);
    p.off_s = take(4 * states), p.off_g = take(4 * states);
    p.off_sums = take(4 * (uint64_t)(2 * p.chunks * f.B * f.H));
    const DeltaPlan forward = delta_plan(f);
    p.off_forward = take(forward.bytes);
    p.off_grads = take(4 * (uint64_t)(forward.segments > 1 ? forward.segments - 1 : 0) * (uint64_t)(f.B * f.H * f.V * f.K));
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
    const DeltaKept kept = {at(plan.off_u), at(plan.off_s), plan.Vp}, back = {at(plan.off_du), at(plan.off_g), plan.Vp};
    int32_t st;
    if (plan.tokens) {
        st = launch_delta_tokens(in, kept, stream);
        if (st == kOk)
            st = launch_delta_tokens_bwd(a, back, stream);
    } else {
        const DeltaPlan forward = delta_plan(f);
        st = launch_delta_prepare(in, ws + plan.off_forward + forward.off_prepared, stream);
        if (st == kOk)
            st = launch_delta_chunks(in, forward, ws + plan.off_forward, kept, stream);
        if (st == kOk)
            st = launch_delta_chunks_bwd(a, forward, ws + plan.off_forward, at(plan.off_grads), back, stream);
    }
    if (st != kOk)
        return st;
    GradParams p = {};
    p.d = delta_params(in);
    p.d.grad_y = static_cast<const uint16_t *>(a.grad_y);
    for (int i = 0; i < 3; ++i)
        p.d.gy_s[i] = a.grad_y_strides[i];
    p.u = kept.u, p.du = back.u, p.s = kept.states, p.g = back.states, p.Vp = plan.Vp;
    const auto vectors = [&](const void *x, const int64_t (&s)[3]) { return vectors_for(f.V, (uintptr_t)x, s[0] | s[1] | s[2]); };
    p.vectors_gy = vectors(a.grad_y, a.grad_y_strides), p.vectors_v = vectors(f.v, f.v_strides);
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
