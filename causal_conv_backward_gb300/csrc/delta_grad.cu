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
// All products are on the tensor cores, of fp16 operands: two terms (22 bits) of
// fp32 rows scaled by a power of two, q and k exact in one. A tile of 64 values
// of V at a time, the rows of grad_y and du are multiplied with those of S and u,
// the rows of u with those of G; then the tokens' own products follow. A thread
// has one token's row, of grad_y (P', gq') or of du and u (L', gk'), and a quarter
// of the columns; sums over tiles and heads are fp32 in its registers. What
// bounds the kernel is reading u, du, S and G, 4 bytes a value, and their rounding,
// and that a block's phases (loads, terms, products, sums) follow on one another:
// shared memory and tensor memory hold one tile. 2048 tokens of 8 x 16 heads of
// 128 x 128 take 623 us; their 1.2 GB would take 180, the products 100.
#include "delta_common.cuh"
#include "tensor_core.cuh"

namespace mcc1d {

namespace {

constexpr int kC = kChunk, kVT = 64, kThreads = 512, kQuarters = 4;

struct GradParams {
    DeltaParams d;
    const float *u, *du, *s, *g;   // [S,B,H,Vp], [chunks][B H][K,Vp]
    int32_t Vp;
    bool vectors_q, vectors_k, vectors_gy, vectors_v, vectors_out;
    uint16_t *grad_q, *grad_k, *grad_delta, *grad_beta;
    float *sum_A, *sum_bias;       // [chunks B][H]
};

// Operands in shared memory. Panels of rows along V: grad_y, du, u (64 rows each,
// one after the other), S and G (a row to a key); later rows along the tokens:
// P' and L' (64 rows each), and the two that are taken by columns.
template <int KP>
struct Panels {
    static constexpr int kRows = 3 * kPanelBytes;                   // of grad_y, du, u
    static constexpr int kKeys = KP * 128;
    static constexpr int A = 0, ALo = kRows, S = 2 * kRows, SLo = S + kKeys, G = S + 2 * kKeys, GLo = S + 3 * kKeys, QK = S + 4 * kKeys;
    static constexpr int kQK = 2 * kPanelBytes;                     // rows of q, then of k, 64 keys of them
    static constexpr int kBytes = QK + KP / 64 * kQK;
    static constexpr int X = A, XLo = ALo, PC = S, PCLo = S + kPanelBytes, LC = S + 2 * kPanelBytes, LCLo = S + 3 * kPanelBytes;
};

struct GradShared {
    uint64_t done;
    uint32_t tmem;
    float of_rows[3 * kC], of_s[128], of_g[128];                     // what operands are multiplied by
    float ch[kC], cl[kC], b[kC], dt[kC], raw[kC], fq[kC], fk[kC];    // fq, fk: of q, k as they are
    float xq[kC], xk[kC];                                           // of q, k as operands
    float gc[kC], gb[kC], dv[kC], dot[kThreads / 32];
    float dots[3][kQuarters][kC], low[kQuarters][kC];
    float cross[2][kQuarters][kC], later[2][kC / 2];                 // sums over decayed pairs
    float most[kQuarters][2 * kC];
    float4 most_col[kC];                                             // of the four warps of a column
};

// Columns of tensor memory: [grad_y; du] S, [grad_y; du] u, [du; u] G, [q; k] k;
// then [P'; L'] k in G's place and the column products in S's.
enum { kDS = 0, kDU = 128, kDG = 192, kDK = 320, kColumns = 512 };

// Eight values of a workspace row, zeros past its end.
__device__ __forceinline__ void load8(const float *from, int live, float (&x)[8])
{
    if (live >= 8) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(from)), w = __ldg(reinterpret_cast<const float4 *>(from) + 1);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w, x[4] = w.x, x[5] = w.y, x[6] = w.z, x[7] = w.w;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e < live)
            v = __ldg(reinterpret_cast<const float4 *>(from + e));
        x[e] = v.x, x[e + 1] = e + 1 < live ? v.y : 0.f, x[e + 2] = e + 2 < live ? v.z : 0.f, x[e + 3] = e + 3 < live ? v.w : 0.f;
    }
}
template <int DT>
__device__ __forceinline__ void load8(const uint16_t *from, bool vectors, int live, float (&x)[8])
{
    if (vectors) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (live > 0)
            v = __ldg(reinterpret_cast<const uint4 *>(from));
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<DT>(u[e]);
            x[2 * e] = f.x, x[2 * e + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = e < live ? value<DT>(from + e) : 0.f;
    }
}
__device__ __forceinline__ float most8(const float (&x)[8])
{
    return fmaxf(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))),
                 fmaxf(fmaxf(fabsf(x[4]), fabsf(x[5])), fmaxf(fabsf(x[6]), fabsf(x[7]))));
}
// The N threads that share a row.
template <int N>
__device__ __forceinline__ float most_of_lanes(float x)
{
#pragma unroll
    for (int d = 1; d < N; d *= 2)
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
    return x;
}
template <int N>
__device__ __forceinline__ float sum_of_lanes(float x)
{
#pragma unroll
    for (int d = 1; d < N; d *= 2)
        x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    return x;
}
__device__ __forceinline__ void put8(uint8_t *hi, uint8_t *lo, uint32_t at, const float *x, float scale)
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        two_terms(make_float2(x[2 * e] * scale, x[2 * e + 1] * scale), h[e], l[e]);
    *reinterpret_cast<uint4 *>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
}
// A row's eight values (of its 64, over eight threads) as terms; 1 / its scale.
__device__ __forceinline__ float put_row(uint8_t *hi, uint8_t *lo, int row, int piece, const float (&x)[8])
{
    const float scale = scale_for(most_of_lanes<8>(most8(x)));
    put8(hi, lo, panel_at(row, piece), x, scale);
    return inverse_scale(scale);
}

// The rows of a tile of V, asked for ahead of their use (64 values of a row are
// two lines of 128 bytes; a thread of every four asks).
__device__ __forceinline__ void ask_ahead(const GradParams &gp, int64_t chunk, int64_t item, int v0, int row, int piece, int n)
{
    const DeltaParams &p = gp.d;
    const int at = v0 + 8 * piece;
    if (piece % 4 || at >= p.V)
        return;
    const auto ask = [](const float *x) { asm volatile("prefetch.global.L2 [%0];" ::"l"(x)); };
    const int64_t BH = (int64_t)p.B * p.H;
    if (row < n) {
        const int64_t from = ((chunk * kC + row) * BH + item) * gp.Vp + at;
        ask(gp.u + from), ask(gp.du + from);
    }
    for (int k = row; k < p.K; k += kC) {
        const int64_t from = ((chunk * BH + item) * p.K + k) * gp.Vp + at;
        ask(gp.s + from), ask(gp.g + from);
    }
}

// Sums (or the largest) of 16 values over the warp's lanes: lane l has that of value l / 2.
template <class F>
__device__ __forceinline__ float of16(float (&x)[16], F &&join)
{
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int d = 16, n = 8; n > 0; d /= 2, n /= 2) {
        const bool upper = lane & d;
#pragma unroll
        for (int e = 0; e < n; ++e) {
            const float give = upper ? x[e] : x[e + n], keep = upper ? x[e + n] : x[e];
            x[e] = join(keep, __shfl_xor_sync(0xFFFFFFFFu, give, d));
        }
    }
    return join(x[0], __shfl_xor_sync(0xFFFFFFFFu, x[0], 1));
}
// A sum over this lane and those after it.
__device__ __forceinline__ float from_lane_on(float x)
{
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const float o = __shfl_down_sync(0xFFFFFFFFu, x, d);
        if (threadIdx.x % 32 + d < 32)
            x += o;
    }
    return x;
}

// Adds A B^T, all of two terms but A's second times B's second, over 64 values
// of the sum, by one thread; second terms first, as in delta_chunks.cu.
__device__ __forceinline__ void three_products(uint32_t d, uint32_t a, uint32_t a_lo, uint32_t b, uint32_t b_lo, uint32_t kind)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        mma_ss(d, desc_rows(a) + 2 * j, desc_rows(b_lo) + 2 * j, kind, j > 0);
        mma_ss(d, desc_rows(a_lo) + 2 * j, desc_rows(b) + 2 * j, kind, true);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        mma_ss(d, desc_rows(a) + 2 * j, desc_rows(b) + 2 * j, kind, true);
}

template <int DT, int KP>
__global__ void __launch_bounds__(kThreads, 1) mcc1d_delta_grad_chunk(const __grid_constant__ GradParams gp)
{
    extern __shared__ uint8_t raw_shared[];
    __shared__ GradShared sh;
    typedef Panels<KP> Pn;
    uint8_t *panels = raw_shared + (1024 - smem_u32(raw_shared) % 1024) % 1024;
    const uint32_t at_panels = smem_u32(panels);
    constexpr int KC = KP / kQuarters, UNIT = 16, IC = kC / kQuarters;        // a thread's keys and other tokens
    const DeltaParams &p = gp.d;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, quarter = warp / 4;
    const int r = 32 * (warp % 4) + lane, t = r % kC;             // its row of a product, and token
    const bool of_du = r >= kC;                                   // a whole warp's
    const int g = blockIdx.x % p.G, b = (blockIdx.x / p.G) % p.B, per = p.H / p.G;
    const int64_t chunk = blockIdx.x / p.G / p.B, t0 = chunk * kC;
    const int64_t length = clamped_length(p.lengths, b, p.S);
    const int there = (int)(p.S - t0 < kC ? p.S - t0 : kC);                            // rows to write
    const int n = (int)(length <= t0 ? 0 : length - t0 < kC ? length - t0 : kC);       // tokens that are there
    const int64_t BH = (int64_t)p.B * p.H;
    const int prow = tid / 8, piece = tid % 8;                    // of the rows on their way to panels

    if (n == 0) {
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
        for (int e = tid; e < there * p.K; e += kThreads) {
            const int64_t at = (((t0 + e / p.K) * p.B + b) * p.G + g) * p.K + e % p.K;
            gp.grad_q[at] = gp.grad_k[at] = 0;
        }
        return;
    }
    if (tid == 0) {
        mbar_init(smem_u32(&sh.done), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    if (warp == 0)
        tmem_alloc(smem_u32(&sh.tmem), kColumns);
    // q and k: as operands, and what they are multiplied by
    {
        float x[2][KP / 64][8];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint16_t *from = w ? p.k + (t0 + prow) * p.k_s[0] + b * p.k_s[1] + g * p.k_s[2] : p.q + (t0 + prow) * p.q_s[0] + b * p.q_s[1] + g * p.q_s[2];
#pragma unroll
            for (int j = 0; j < KP / 64; ++j) {
                const int at = 64 * j + 8 * piece;
                load8<DT>(from + at, w ? gp.vectors_k : gp.vectors_q, prow < n ? p.K - at : 0, x[w][j]);
            }
        }
        ask_ahead(gp, chunk, (int64_t)b * p.H + g * per, 0, prow, piece, n);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            float sum = 0.f, most = 0.f;
#pragma unroll
            for (int j = 0; j < KP / 64; ++j) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum = fmaf(x[w][j][e], x[w][j][e], sum);
                most = fmaxf(most, most8(x[w][j]));
            }
            sum = sum_of_lanes<8>(sum);
            const float scale = scale_for(most_of_lanes<8>(most)), f = unit_factor(p.flags, sum);
#pragma unroll
            for (int j = 0; j < KP / 64; ++j) {
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    h[e] = pack_half2(make_float2(x[w][j][2 * e] * scale, x[w][j][2 * e + 1] * scale));
                *reinterpret_cast<uint4 *>(panels + Pn::QK + j * Pn::kQK + w * kPanelBytes + panel_at(prow, piece)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
            if (piece == 0) {
                if (w)
                    sh.fk[prow] = f, sh.xk[prow] = f * inverse_scale(scale);
                else
                    sh.fq[prow] = f * p.scale, sh.xq[prow] = f * p.scale * inverse_scale(scale);
            }
        }
    }
    shared_to_async();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem, lanes = tmem + ((uint32_t)(32 * (warp % 4)) << 16);
    constexpr uint32_t by_tokens = mma_kind(kC, false), by_keys = mma_kind(KP, false), keys_by_columns = mma_kind(KP, true), both_by_columns = mma_kind(KP, true, true);
    uint32_t parity = 0;
    bool ok = true;          // no wait gave up
    if (tid == 0)            // q.k and k.k, exact; done with the first products that are waited for
#pragma unroll
        for (int j = 0; j < KP / 16; ++j) {
            const uint32_t at = at_panels + Pn::QK + (j / 4) * Pn::kQK;
            mma_ss(tmem + kDK, desc_rows(at) + 2 * (j % 4), desc_rows(at + kPanelBytes) + 2 * (j % 4), by_tokens, j > 0);
        }
    float acc[KC];           // of gq' or gk', over tiles and the heads that share them
#pragma unroll
    for (int c = 0; c < KC; ++c)
        acc[c] = 0.f;
    // this thread's keys of q (or k) as an operand
    const auto own = [&](int c, float2 (&x)[4]) {      // eight from c on
        const int at = quarter * KC + c;
        const uint4 v = *reinterpret_cast<const uint4 *>(panels + Pn::QK + (at / 64) * Pn::kQK + (of_du ? kPanelBytes : 0) + panel_at(t, at % 64 / 8));
        x[0] = unpack2<1>(v.x), x[1] = unpack2<1>(v.y), x[2] = unpack2<1>(v.z), x[3] = unpack2<1>(v.w);
    };

    for (int h = g * per; h < (g + 1) * per; ++h) {
        const int64_t item = (int64_t)b * p.H + h;
        float raw_delta[2] = {0.f, 0.f}, raw_beta[2] = {0.f, 0.f};      // of the first warp's tokens
        if (warp == 0)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t at = t0 + 2 * lane + e;
                if (2 * lane + e < n) {
                    if (p.delta)
                        raw_delta[e] = value<DT>(p.delta + at * p.delta_s[0] + b * p.delta_s[1] + h);
                    raw_beta[e] = value<DT>(p.beta + at * p.beta_s[0] + b * p.beta_s[1] + h);
                }
            }
        __syncthreads();

        float PL[IC], gs = 0.f, dv = 0.f, dot_s = 0.f, dot_g = 0.f;       // P' or L'; sums of S G, du.v, and along the row's q or k
#pragma unroll
        for (int c = 0; c < IC; ++c)
            PL[c] = 0.f;
        for (int v0 = 0; v0 < p.V; v0 += kVT) {
            {
                float x[8], y[8];
                const int at = v0 + 8 * piece, live = prow < n ? p.V - at : 0;
                const int64_t from = ((t0 + prow) * BH + item) * gp.Vp + at;
                const float *s = gp.s + ((chunk * BH + item) * p.K + prow) * gp.Vp + at, *gr = gp.g + (s - gp.s);
                float xs[KP / 64][8], xg[KP / 64][8];
#pragma unroll
                for (int j = 0; j < KP / 64; ++j) {
                    const int there_k = prow + 64 * j < p.K ? p.V - at : 0;
                    load8(s + (int64_t)64 * j * gp.Vp, there_k, xs[j]);
                    load8(gr + (int64_t)64 * j * gp.Vp, there_k, xg[j]);
                }
                load8(gp.du + from, live, x);
                load8<DT>(p.v + (t0 + prow) * p.v_s[0] + b * p.v_s[1] + h * p.v_s[2] + at, gp.vectors_v, live, y);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dv = fmaf(x[e], y[e], dv);
                const float of_du_row = put_row(panels + Pn::A, panels + Pn::ALo, kC + prow, piece, x);
                load8(gp.u + from, live, x);
                load8<DT>(p.grad_y + (t0 + prow) * p.gy_s[0] + b * p.gy_s[1] + h * p.gy_s[2] + at, gp.vectors_gy, live, y);
#pragma unroll
                for (int j = 0; j < KP / 64; ++j) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        gs = fmaf(xs[j][e], xg[j][e], gs);
                    const float of = put_row(panels + Pn::S, panels + Pn::SLo, 64 * j + prow, piece, xs[j]);
                    const float og = put_row(panels + Pn::G, panels + Pn::GLo, 64 * j + prow, piece, xg[j]);
                    if (piece == 0)
                        sh.of_s[64 * j + prow] = of, sh.of_g[64 * j + prow] = og;
                }
                const float of_u_row = put_row(panels + Pn::A, panels + Pn::ALo, 2 * kC + prow, piece, x);
                const float of_y_row = put_row(panels + Pn::A, panels + Pn::ALo, prow, piece, y);
                if (piece == 0)
                    sh.of_rows[prow] = of_y_row, sh.of_rows[kC + prow] = of_du_row, sh.of_rows[2 * kC + prow] = of_u_row;
            }
            if (warp == 0 && v0 == 0) {
                // gates, and the running sum of log2 a in two parts whose differences are
                // exact in the first: multiples of 2^-9 below 2^14
                float hi[2], lo[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * lane + e;
                    Gates gate = {0.f, 0.f, 0.f, 0.f};
                    if (i < n)
                        gate = gates_of(p.flags, p.delta != nullptr, raw_delta[e], p.delta_bias ? __ldg(p.delta_bias + h) : 0.f, p.delta ? __ldg(p.A + h) : 0.f,
                                        raw_beta[e]);
                    const float l = held_log2(gate.log2a);
                    hi[e] = rintf(l * 512.f) * (1.f / 512.f), lo[e] = l - hi[e];
                    sh.b[i] = gate.b, sh.dt[i] = gate.dt, sh.raw[i] = gate.raw;
                }
                float x = hi[0] + hi[1], y = lo[0] + lo[1];
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const float ox = __shfl_up_sync(0xFFFFFFFFu, x, d), oy = __shfl_up_sync(0xFFFFFFFFu, y, d);
                    if (lane >= d)
                        x += ox, y += oy;
                }
                sh.ch[2 * lane] = x - hi[1], sh.ch[2 * lane + 1] = x;
                const float before = __shfl_up_sync(0xFFFFFFFFu, y, 1);
                sh.cl[2 * lane] = (lane > 0 ? before : 0.f) + lo[0], sh.cl[2 * lane + 1] = y;
            }
            shared_to_async();
            tmem_fence_before();
            __syncthreads();
            tmem_fence_after();
            if (v0 + kVT < p.V)
                ask_ahead(gp, chunk, item, v0 + kVT, prow, piece, n);
            else if (h + 1 < (g + 1) * per)
                ask_ahead(gp, chunk, item + 1, 0, prow, piece, n);
            if (tid == 0) {
                three_products(tmem + kDS, at_panels + Pn::A, at_panels + Pn::ALo, at_panels + Pn::S, at_panels + Pn::SLo, by_keys);
                three_products(tmem + kDU, at_panels + Pn::A, at_panels + Pn::ALo, at_panels + Pn::A + 2 * kPanelBytes, at_panels + Pn::ALo + 2 * kPanelBytes,
                               by_tokens);
                three_products(tmem + kDG, at_panels + Pn::A + kPanelBytes, at_panels + Pn::ALo + kPanelBytes, at_panels + Pn::G, at_panels + Pn::GLo, by_keys);
                mma_commit(smem_u32(&sh.done));
            }
            ok = ok && mbar_wait_bounded(smem_u32(&sh.done), parity);
            parity ^= 1;
            tmem_fence_after();
            __syncwarp();
            const float of_row = sh.of_rows[r], bt = sh.b[t];
            const float ec = ex2_held(sh.ch[t] + sh.cl[t]), el = ex2_held((sh.ch[kC - 1] - sh.ch[t]) + (sh.cl[kC - 1] - sh.cl[t]));
            const float add = (of_du ? -ec : ec) * of_row, to_acc = of_du ? bt : 1.f, add_g = of_du ? el * sh.of_rows[kC + r] : 0.f;
#pragma unroll
            for (int c = 0; c < KC; c += UNIT) {
                uint32_t d[UNIT];
                tmem_load(lanes + kDS + quarter * KC + c, d);
                tmem_wait(d);
#pragma unroll
                for (int e = 0; e < UNIT; e += 8) {
                    float2 x[4];
                    own(c + e, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float y = __uint_as_float(d[e + i]) * (add * sh.of_s[quarter * KC + c + e + i]);
                        dot_s = fmaf(y, i % 2 ? x[i / 2].y : x[i / 2].x, dot_s);
                        acc[c + e + i] = fmaf(to_acc, y, acc[c + e + i]);
                    }
                }
            }
            if (of_du)
#pragma unroll
                for (int c = 0; c < KC; c += UNIT) {
                    uint32_t d[UNIT];
                    tmem_load(lanes + kDG + quarter * KC + c, d);
                    tmem_wait(d);
#pragma unroll
                    for (int e = 0; e < UNIT; e += 8) {
                        float2 x[4];
                        own(c + e, x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float y = __uint_as_float(d[e + i]) * (add_g * sh.of_g[quarter * KC + c + e + i]);
                            dot_g = fmaf(y, i % 2 ? x[i / 2].y : x[i / 2].x, dot_g);
                            acc[c + e + i] += y;
                        }
                    }
                }
            {
                uint32_t d[IC];
                tmem_load(lanes + kDU + quarter * IC, d);
                tmem_wait(d);
                const float f = of_du ? -of_row : of_row;
#pragma unroll
                for (int c = 0; c < IC; ++c)
                    PL[c] = fmaf(__uint_as_float(d[c]), f * sh.of_rows[2 * kC + quarter * IC + c], PL[c]);
            }
            tmem_fence_before();
            __syncthreads();
        }
        gs = sum_of_lanes<32>(gs);
        if (lane == 0)
            sh.dot[warp] = gs;
        dv = sum_of_lanes<8>(dv);
        if (piece == 0)
            sh.dv[prow] = dv;
        if (of_du) {
            sh.dots[1][quarter][t] = dot_s * sh.xk[t];
            sh.dots[2][quarter][t] = dot_g * sh.xk[t];
        } else {
            sh.dots[0][quarter][t] = dot_s * sh.xq[t];
        }
        // P' and L', with the decays; by rows for the products with k, by columns
        // with what the row's own token is multiplied by
        {
            uint32_t d[IC];
            tmem_load(lanes + kDK + quarter * IC, d);
            tmem_wait(d);
            float E[IC], by_row[IC], low = 0.f, most_row = 0.f;
            const float th = sh.ch[t], tl = sh.cl[t], f = of_du ? sh.xk[t] : sh.xq[t], bt = of_du ? sh.b[t] : 1.f;
#pragma unroll
            for (int c = 0; c < IC; ++c) {
                const int i = quarter * IC + c;
                const bool in = of_du ? i < t : i <= t;
                const float D = in ? ex2_held((th - sh.ch[i]) + (tl - sh.cl[i])) : 0.f, x = in ? PL[c] * D : 0.f;
                const float xi = sh.xk[i], lk = x * (__uint_as_float(d[c]) * f * xi);
                E[c] = i < t ? bt * lk : 0.f;      // no decay between a token and itself
                low += lk;
                by_row[c] = bt * x * xi;
                PL[c] = bt * x * f;
                most_row = fmaxf(most_row, fabsf(by_row[c]));
            }
            // The pairs (t, i) whose decay a token has part in are those with i before it and t
            // not. Only they are summed: pairs behind it, however much larger, would leave
            // their rounding. A warp has 32 t and 16 i; behind all of its i a token has
            // the whole rows from it on, within them those rows' sums up to it.
            {
                const bool within = quarter / 2 == warp % 2;
                const auto sum = [](float x, float y) { return x + y; };
                float rows = 0.f;
                if (within) {
#pragma unroll
                    for (int c = 0; c < IC; ++c) {
                        rows += E[c];
                        E[c] = t > quarter * IC + c ? rows : 0.f;      // for the token after c
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < IC; ++c)
                        rows += E[c];
                }
                rows = from_lane_on(rows);
                const float sums = of16(E, sum);
                const int at = quarter * IC + lane / 2;
                if (!within || t <= quarter * IC || t > quarter * IC + IC)
                    sh.cross[of_du][quarter][t] = quarter * IC < t ? rows : 0.f;
                if (lane % 2 == 0 && within && (at + 1) / 32 == warp % 2)
                    sh.cross[of_du][quarter][at + 1] = sums;
                if (lane % 2 == 0 && quarter / 2 < warp % 2)           // of tokens in the other half
                    sh.later[of_du][at] = sums;
            }
            if (of_du)
                sh.low[quarter][t] = low;
            // a column's pairs, of rows that P' and L' fade or grow along, are a sum of their own
#pragma unroll
            for (int c = 0; c < IC; ++c)
                E[c] = fabsf(PL[c]);
            const float most_col = of16(E, [](float x, float y) { return fmaxf(x, y); });
            if (lane % 2 == 0)
                reinterpret_cast<float *>(&sh.most_col[quarter * IC + lane / 2])[warp % 4] = most_col;
            sh.most[quarter][r] = most_row;
            tmem_fence_before();
            __syncthreads();
            tmem_fence_after();
            most_row = fmaxf(fmaxf(sh.most[0][r], sh.most[1][r]), fmaxf(sh.most[2][r], sh.most[3][r]));
            const auto scale_of = [&](int i) {
                const float4 m = sh.most_col[i];
                return scale_for(fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w)));
            };
            const float scale_row = scale_for(most_row), scale_lane = scale_of(quarter * IC + lane % IC);
#pragma unroll
            for (int c = 0; c < IC; ++c)
                PL[c] *= __shfl_sync(0xFFFFFFFFu, scale_lane, c);
            uint8_t *hi = panels + (of_du ? Pn::LC : Pn::PC), *lo = panels + (of_du ? Pn::LCLo : Pn::PCLo);
#pragma unroll
            for (int e = 0; e < IC / 8; ++e) {
                put8(panels + Pn::X, panels + Pn::XLo, panel_at(r, quarter * (IC / 8) + e), by_row + 8 * e, scale_row);
                put8(hi, lo, panel_at(t, quarter * (IC / 8) + e), PL + 8 * e, 1.f);
            }
            shared_to_async();
            tmem_fence_before();
            __syncthreads();
            tmem_fence_after();
            if (tid == 0) {
                const uint32_t qk = at_panels + Pn::QK;
#pragma unroll
                for (int lo = 1; lo >= 0; --lo)
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j) {
                        const uint64_t step = (uint64_t)(2048 * j >> 4);
                        const uint64_t q = desc_columns(qk, Pn::kQK) + step, k = desc_columns(qk + kPanelBytes, Pn::kQK) + step;
                        const bool add = !lo || j > 0;
                        mma_ss(tmem + kDG, desc_rows(at_panels + (lo ? Pn::XLo : Pn::X)) + 2 * j, k, keys_by_columns, add);
                        // 128 columns to the product, of the panel before too: the second half's rows are read
                        mma_ss(tmem + kDS, desc_columns(at_panels + (lo ? Pn::PCLo : Pn::PC) - kPanelBytes, kPanelBytes) + step, q, both_by_columns, add);
                        mma_ss(tmem + kDS, desc_columns(at_panels + (lo ? Pn::LCLo : Pn::LC) - kPanelBytes, kPanelBytes) + step, k, both_by_columns, true);
                    }
                mma_commit(smem_u32(&sh.done));
            }
            ok = ok && mbar_wait_bounded(smem_u32(&sh.done), parity);
            parity ^= 1;
            tmem_fence_after();
            __syncwarp();
            const float of_x = inverse_scale(scale_row), of_c = of_du ? inverse_scale(scale_of(t)) : 0.f;
#pragma unroll
            for (int c = 0; c < KC; c += UNIT) {
                uint32_t x[UNIT], y[UNIT];
                tmem_load(lanes + kDG + quarter * KC + c, x);
                tmem_load(lanes + kDS + quarter * KC + c, y);
                tmem_wait(x), tmem_wait(y);
#pragma unroll
                for (int e = 0; e < UNIT; ++e) {
                    acc[c + e] = fmaf(of_x, __uint_as_float(x[e]), acc[c + e]);
                    if (of_du)
                        acc[c + e] = fmaf(of_c, __uint_as_float(y[e]), acc[c + e]);
                }
            }
            tmem_fence_before();
        }
        if (warp == 0) {
            const float A = p.delta ? __ldg(p.A + h) : 0.f;
            const auto four = [](const float (&x)[kQuarters][kC], int i) { return (x[0][i] + x[1][i]) + (x[2][i] + x[3][i]); };
            // of pairs; of the end's products, which have the decays after their token; and
            // of all others, which have those up to theirs
            float pairs[2], x[2], e_of[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                pairs[e] = four(sh.cross[0], i) + four(sh.cross[1], i);
                const float sk = four(sh.dots[1], i);
                e_of[e] = four(sh.dots[2], i);
                x[e] = four(sh.dots[0], i) + sh.b[i] * sk;
                sh.gb[i] = sh.dv[i] + sk + four(sh.low, i);
                if (!ok)
                    x[e] = sh.gb[i] = __uint_as_float(0x7FFFFFFFu);
            }
            {       // tokens of the first half: the second half's pairs with those before them
                const int i = 2 * lane;
                const float l0 = lane < 16 ? sh.later[0][i] + sh.later[1][i] : 0.f, l1 = lane < 16 ? sh.later[0][i + 1] + sh.later[1][i + 1] : 0.f;
                float to = l0 + l1;
#pragma unroll
                for (int d = 1; d < 16; d *= 2) {
                    const float o = __shfl_up_sync(0xFFFFFFFFu, to, d);
                    if (lane >= d)
                        to += o;
                }
                const float o = __shfl_up_sync(0xFFFFFFFFu, to, 1), before = lane > 0 ? o : 0.f;
                if (lane < 16)
                    pairs[0] += before, pairs[1] += before + l0;
            }
            if (lane == 31) {
                float s = 0.f;
                for (int w = 0; w < kThreads / 32; ++w)
                    s += sh.dot[w];
                x[1] = fmaf(s, ex2_held(sh.ch[kC - 1] + sh.cl[kC - 1]), x[1]);
            }
            float s = x[0] + x[1], s_e = e_of[0] + e_of[1];
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const float o = __shfl_down_sync(0xFFFFFFFFu, s, d), oe = __shfl_up_sync(0xFFFFFFFFu, s_e, d);
                if (lane + d < 32)
                    s += o;
                if (lane >= d)
                    s_e += oe;
            }
            const float o = __shfl_down_sync(0xFFFFFFFFu, s, 1), after = lane < 31 ? o : 0.f;
            const float oe = __shfl_up_sync(0xFFFFFFFFu, s_e, 1), before = lane > 0 ? oe : 0.f;
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                float gl = e ? after + x[1] + (before + e_of[0]) : after + (x[0] + x[1]) + before;
                gl = i < n ? gl + pairs[e] : 0.f;
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
            sa = sum_of_lanes<32>(sa), sb = sum_of_lanes<32>(sb);
            if (lane == 0) {
                gp.sum_A[(chunk * p.B + b) * p.H + h] = sa;
                gp.sum_bias[(chunk * p.B + b) * p.H + h] = sb;
            }
        }
    }
    // through the division by the lengths: (g - x (x.g)) f for a unit vector x
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < KC; c += 8) {
        float2 x[4];
        own(c, x);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dot = fmaf(acc[c + i], i % 2 ? x[i / 2].y : x[i / 2].x, dot);
    }
    __syncthreads();
    sh.most[quarter][r] = dot;
    __syncthreads();
    const float f = of_du ? sh.fk[t] : sh.fq[t], fx = of_du ? sh.xk[t] : sh.xq[t];
    dot = (sh.most[0][r] + sh.most[1][r]) + (sh.most[2][r] + sh.most[3][r]);
    // q' is scale times a unit vector
    const float along = of_du ? fx : p.scale != 0.f ? fx / p.scale : 0.f;
    const float back = p.flags & MCC1D_QK_NORM ? -dot * along * along : 0.f;
    if (t < there) {
        uint16_t *to = (of_du ? gp.grad_k : gp.grad_q) + (((t0 + t) * p.B + b) * p.G + g) * p.K;
#pragma unroll
        for (int c = 0; c < KC; c += 8) {
            float2 x[4];
            own(c, x);
            const int at = quarter * KC + c;
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 v = make_float2(fmaf(back, x[i].x, acc[c + 2 * i]) * f, fmaf(back, x[i].y, acc[c + 2 * i + 1]) * f);
                if (!ok)
                    v.x = v.y = __uint_as_float(0x7FFFFFFFu);
                u[i] = pack2<DT>(v);
            }
            if (gp.vectors_out) {
                if (at < p.K)
                    *reinterpret_cast<uint4 *>(to + at) = make_uint4(u[0], u[1], u[2], u[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (at + i < p.K)
                        to[at + i] = (uint16_t)(u[i / 2] >> (16 * (i % 2)));
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 0) {
        tmem_fence_after();
        tmem_free(tmem, kColumns);
    }
}

template <int DT, int KP>
int32_t grad(const GradParams &p, int64_t blocks, cudaStream_t stream)
{
    constexpr int bytes = Panels<KP>::kBytes + 1024;
    if (cudaFuncSetAttribute(mcc1d_delta_grad_chunk<DT, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return kErrCuda;
    return launch(mcc1d_delta_grad_chunk<DT, KP>, dim3((unsigned)blocks), kThreads, bytes, stream, p);
}

}  // namespace

DeltaBwdPlan delta_bwd_plan(const mcc1d_delta_bwd_args &a)
{
    const mcc1d_delta_args &f = a.fwd;
    DeltaBwdPlan p = {};
    p.chunks = (f.S + kChunk - 1) / kChunk;
    p.Vp = (int32_t)((f.V + 3) / 4 * 4);
    p.tokens = delta_plan(f, true).tokens;
    const auto take = [&](uint64_t bytes) {
        const uint64_t at = p.bytes;
        p.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    const uint64_t tokens = (uint64_t)(f.S * f.B * f.H) * p.Vp, states = (uint64_t)(p.chunks * f.B * f.H * f.K) * p.Vp;
    p.off_u = take(4 * tokens), p.off_du = take(4 * tokens);
    p.off_s = take(4 * states), p.off_g = take(4 * states);
    p.off_sums = take(4 * (uint64_t)(2 * p.chunks * f.B * f.H));
    const DeltaPlan forward = delta_plan(f, true);
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
        const DeltaPlan forward = delta_plan(f, true);
        st = launch_delta_prepare(in, ws + plan.off_forward + forward.off_prepared, true, stream);
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
    const auto vectors = [](int64_t n, const void *x, const int64_t (&s)[3]) { return vectors_for(n, (uintptr_t)x, s[0] | s[1] | s[2]); };
    p.vectors_gy = vectors(f.V, a.grad_y, a.grad_y_strides), p.vectors_v = vectors(f.V, f.v, f.v_strides);
    p.vectors_q = vectors(f.K, f.q, f.q_strides), p.vectors_k = vectors(f.K, f.k, f.k_strides);
    p.vectors_out = vectors_for(f.K, (uintptr_t)a.grad_q | (uintptr_t)a.grad_k, 0);
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
