// ssm_scan_bwd.cu - gradients of the selective scan.
//
// With g(t) the gradient that reaches the state h(t) and dy the gradient of y
// before the gate:
//
//   g(t)[n]  = C(t)[n] dy(t) + a(t+1)[n] g(t+1)[n],   a(t) = exp(dt A)
//   q(t)[n]  = g(t)[n] a(t)[n] h(t-1)[n]
//   grad_C   = sum over the group's channels of dy h,   grad_B = sum of g dt u
//   grad_u   = dt sum_n g B + D dy
//   grad_dt  = sum_n A q + u sum_n g B,   grad_A = sum over b, t of dt q
//
// A first pass (mcc1d_ssm_scan, kSummaryGrad) leaves the state at every tile
// start and, per time chunk, what the join needs to give each chunk its
// incoming state and incoming gradient; all chunks then run at once. A block
// walks its chunk's tiles backwards. In a tile the states are run forward
// again, kept every kSub rows in shared memory, and each run of kSub rows is
// computed once more with its states and decays in registers for the
// recurrence back. Sums over a channel's states and over a warp's channels go
// through shuffles, those over warps and blocks through memory, in a fixed
// order.
#include "plan.h"
#include "ssm_scan.cuh"

namespace mcc1d {

namespace {

constexpr int kSub = 4, kBwdWarps = BwdTile<1>::WARPS, kThreads = 32 * kBwdWarps;

template <int NL>
struct BwdShared {
    using T = BwdTile<NL>;
    static constexpr int TT = T::TT;
    float4 sq[TT][T::CB];                         // dt, dt u, dy -> sum A q, sum g B, y; dt
    float4 hs[TT / kSub][kThreads];           // states before each run of kSub rows
    float sB[TT][T::NP], sC[TT][T::NP];
    float bc[TT][kBwdWarps][2 * T::NP];          // a warp's grad_B and grad_C
};

// Sums v[0..K-1] over NL lanes whose numbers 0..NL-1 are the lane bits from
// `bit` up; K and NL are powers of two. Each exchange halves what a lane
// carries on, so K values cost K (1 - 1/NL) shuffles where K >= NL, not
// K log2 NL. Lane number j is left with v[0..] = the sums of values
// j K/NL .. (K >= NL), or with v[0] = that of value j % K (K < NL).
template <int K, int NL>
__device__ __forceinline__ void lanes_sum(float (&v)[K], int lane, int bit)
{
    constexpr int M = K < NL ? K : NL;
    int n = K;
#pragma unroll
    for (int step = M / 2; step >= 1; step /= 2) {
        const bool up = (lane & (step * bit)) != 0;
        n /= 2;
#pragma unroll
        for (int i = 0; i < K / 2; ++i)
            if (i < n) {
                const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, step * bit);
            }
    }
#pragma unroll
    for (int step = M; step < NL; step *= 2)
        v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], step * bit);
}

template <int DT, int NL, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 2) mcc1d_ssm_scan_bwd(const ScanParams p)
{
    using T = BwdTile<NL>;
    using Sh = BwdShared<NL>;
    constexpr int NP = T::NP, CW = T::CL, TT = Sh::TT, RP = T::RP;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Sh &sh = *reinterpret_cast<Sh *>(raw_shared);

    const ScanWhere w = scan_where<T>(p);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = lane % NL, n0 = 4 * j, ci = lane / NL;
    const int cl = warp * CW + ci;
    const int64_t te = clamped_length(p.lengths, w.b, p.S);
    const int pc = 2 * (threadIdx.x % T::CP), pr = threadIdx.x / T::CP;
    const bool on0 = pc < w.nc, on1 = pc + 1 < w.nc;
    const int64_t ch = w.c0 + (on0 ? pc : 0);
    const uint16_t *u = p.u + w.b * p.ub + ch, *delta = p.delta + w.b * p.db + ch;
    const uint16_t *z = p.z ? p.z + w.b * p.zb + ch : nullptr, *gy = p.gy + w.b * p.gb + ch;
    const uint16_t *Bm = p.Bm + w.b * p.Bb + w.g * p.Bg, *Cm = p.Cm + w.b * p.Cb + w.g * p.Cg;
    const float bias0 = p.dbias && on0 ? p.dbias[ch] : 0.f, bias1 = p.dbias && on1 ? p.dbias[ch + 1] : 0.f;
    const float D0 = p.D && on0 ? p.D[ch] : 0.f, D1 = p.D && on1 ? p.D[ch + 1] : 0.f;

    const bool live = cl < w.nc;
    const int64_t hc = w.c0 + (live ? cl : 0);
    const int64_t at = (w.chunk * p.B + w.b) * p.H + hc;
    float2 A[2], A2[2], X[2], gA[2], hin[2];
    {
        const float4 a = load_states(p.A + hc * p.N, n0, p.N, p.vecA);
        A[0] = make_float2(a.x, a.y);
        A[1] = make_float2(a.z, a.w);
        A2[0] = make_float2(a.x * kLog2e, a.y * kLog2e);
        A2[1] = make_float2(a.z * kLog2e, a.w * kLog2e);
        const float4 x = *reinterpret_cast<const float4 *>(p.r + at * NP + n0);
        X[0] = make_float2(x.x, x.y);
        X[1] = make_float2(x.z, x.w);
        const float4 s = *reinterpret_cast<const float4 *>(p.e + at * NP + n0);
        hin[0] = make_float2(s.x, s.y);
        hin[1] = make_float2(s.z, s.w);
        gA[0] = gA[1] = make_float2(0.f, 0.f);
    }
    float2 gD = make_float2(0.f, 0.f), gbias = make_float2(0.f, 0.f);

    const int64_t tile0 = w.chunk * p.tiles_per_chunk;
    const int64_t tile1 = tile0 + p.tiles_per_chunk < p.tiles ? tile0 + p.tiles_per_chunk : p.tiles;
    for (int64_t tile = tile1 - 1; tile >= tile0; --tile) {
        const int64_t t0 = tile * TT;
        if (t0 >= te) {
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                const int64_t t = t0 + pr + r * T::RG;
                if (t < p.S) {
                    const int64_t o = (t * p.B + w.b) * p.H + ch;
                    store_pair<PAIRS>(p.gu + o, 0u, on0, on1);
                    store_pair<PAIRS>(p.gdelta + o, 0u, on0, on1);
                    if (p.gz)
                        store_pair<PAIRS>(p.gz + o, 0u, on0, on1);
                }
            }
            continue;
        }
        uint32_t ru[RP], rd[RP], rz[RP], rg[RP];
        {
            BcTile<T, true> bc;
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                const int64_t t = t0 + pr + r * T::RG;
                const bool ok = t < te;
                ru[r] = load_pair<PAIRS>(u + t * p.us, ok && on0, ok && on1);
                rd[r] = load_pair<PAIRS>(delta + t * p.ds, ok && on0, ok && on1);
                rz[r] = z ? load_pair<PAIRS>(z + t * p.zs, ok && on0, ok && on1) : 0u;
                rg[r] = load_pair<PAIRS>(gy + t * p.gs, ok && on0, ok && on1);
            }
            bc.load(p, Bm + t0 * p.Bs, Cm + t0 * p.Cs, (int)(te - t0 < TT ? te - t0 : TT));
            bc.template put<DT>(p, sh.sB, sh.sC);
        }
#pragma unroll
        for (int r = 0; r < RP; ++r) {
            const int64_t t = t0 + pr + r * T::RG;
            const float2 uv = unpack2<DT>(ru[r]);
            float2 dt = add2(unpack2<DT>(rd[r]), make_float2(bias0, bias1)), g = unpack2<DT>(rg[r]);
            if (p.softplus)
                dt = softplus2(dt);
            if (t >= te)
                dt = make_float2(0.f, 0.f);
            if (z) {
                const float2 zv = unpack2<DT>(rz[r]);
                g.x *= zv.x * sigmoid(zv.x);
                g.y *= zv.y * sigmoid(zv.y);
            }
            sh.sq[pr + r * T::RG][pc] = make_float4(dt.x, dt.x * uv.x, g.x, dt.x);
            sh.sq[pr + r * T::RG][pc + 1] = make_float4(dt.y, dt.y * uv.y, g.y, dt.y);
        }
        // the state at the tile's start: from the chunk's zero start, and what entered the chunk
        float2 h[2];
        {
            const int64_t ct = (tile * p.B + w.b) * p.H + hc;
            const float4 s = *reinterpret_cast<const float4 *>(p.cp + ct * NP + n0);
            const float d = p.cpdt[ct];
            h[0].x = fmaf(ex2(d * A2[0].x), hin[0].x, s.x);
            h[0].y = fmaf(ex2(d * A2[0].y), hin[0].y, s.y);
            h[1].x = fmaf(ex2(d * A2[1].x), hin[1].x, s.z);
            h[1].y = fmaf(ex2(d * A2[1].y), hin[1].y, s.w);
        }
        __syncthreads();
        for (int s = 0; s < TT; s += kSub) {
            sh.hs[s / kSub][threadIdx.x] = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
            if (s + kSub == TT)
                break;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const float2 dd = *reinterpret_cast<const float2 *>(&sh.sq[s + i][cl]);
                const float4 bv = *reinterpret_cast<const float4 *>(&sh.sB[s + i][n0]);
                const float2 dt2 = make_float2(dd.x, dd.x), du2 = make_float2(dd.y, dd.y);
                const float2 a0 = decay2(dt2, A2[0]), a1 = decay2(dt2, A2[1]);
                h[0] = fma2(a0, h[0], mul2(du2, make_float2(bv.x, bv.y)));
                h[1] = fma2(a1, h[1], mul2(du2, make_float2(bv.z, bv.w)));
            }
        }
        float2 tA[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};   // the tile's part of grad_A: short sums first
        for (int s = TT - kSub; s >= 0; s -= kSub) {
            float2 hh[kSub + 1][2], aa[kSub][2];
            float ys[kSub], sa[kSub], sb[kSub];
            {
                const float4 v = sh.hs[s / kSub][threadIdx.x];
                hh[0][0] = make_float2(v.x, v.y);
                hh[0][1] = make_float2(v.z, v.w);
            }
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const float2 dd = *reinterpret_cast<const float2 *>(&sh.sq[s + i][cl]);
                const float4 bv = *reinterpret_cast<const float4 *>(&sh.sB[s + i][n0]);
                const float4 cv = *reinterpret_cast<const float4 *>(&sh.sC[s + i][n0]);
                const float2 dt2 = make_float2(dd.x, dd.x), du2 = make_float2(dd.y, dd.y);
                aa[i][0] = decay2(dt2, A2[0]);
                aa[i][1] = decay2(dt2, A2[1]);
                hh[i + 1][0] = fma2(aa[i][0], hh[i][0], mul2(du2, make_float2(bv.x, bv.y)));
                hh[i + 1][1] = fma2(aa[i][1], hh[i][1], mul2(du2, make_float2(bv.z, bv.w)));
                const float2 y = fma2(hh[i + 1][0], make_float2(cv.x, cv.y), mul2(hh[i + 1][1], make_float2(cv.z, cv.w)));
                ys[i] = y.x + y.y;
            }
#pragma unroll
            for (int i = kSub - 1; i >= 0; --i) {
                const float4 dd = sh.sq[s + i][cl];
                const float4 bv = *reinterpret_cast<const float4 *>(&sh.sB[s + i][n0]);
                const float4 cv = *reinterpret_cast<const float4 *>(&sh.sC[s + i][n0]);
                const float2 dt2 = make_float2(dd.x, dd.x), du2 = make_float2(dd.y, dd.y), dy2 = make_float2(dd.z, dd.z);
                const float2 g0 = fma2(dy2, make_float2(cv.x, cv.y), X[0]), g1 = fma2(dy2, make_float2(cv.z, cv.w), X[1]);
                const float2 b2 = fma2(g0, make_float2(bv.x, bv.y), mul2(g1, make_float2(bv.z, bv.w)));
                sb[i] = b2.x + b2.y;
                X[0] = mul2(aa[i][0], g0);
                X[1] = mul2(aa[i][1], g1);
                const float2 q0 = mul2(X[0], hh[i][0]), q1 = mul2(X[1], hh[i][1]);
                const float2 a2 = fma2(A[0], q0, mul2(A[1], q1));
                sa[i] = a2.x + a2.y;
                tA[0] = fma2(dt2, q0, tA[0]);
                tA[1] = fma2(dt2, q1, tA[1]);
                const float2 v0 = mul2(g0, du2), v1 = mul2(g1, du2);
                const float2 c0 = mul2(hh[i + 1][0], dy2), c1 = mul2(hh[i + 1][1], dy2);
                float v[8] = {v0.x, v0.y, v1.x, v1.y, c0.x, c0.y, c1.x, c1.y};
                lanes_sum<8, CW>(v, lane, NL);
                constexpr int KEEP = CW >= 8 ? 1 : 8 / CW;
                if (ci < 8) {
                    const int k = (ci * KEEP) % 8;      // v[0..KEEP-1] are values k.. of the eight
                    float *o = &sh.bc[s + i][warp][(k / 4) * NP + n0 + k % 4];
#pragma unroll
                    for (int m = 0; m < KEEP; ++m)
                        o[m] = v[m];
                }
            }
            lanes_sum<kSub, NL>(ys, lane, 1);
            lanes_sum<kSub, NL>(sa, lane, 1);
            lanes_sum<kSub, NL>(sb, lane, 1);
            constexpr int OWN = NL >= kSub ? 1 : kSub / NL;
            if (j < kSub) {
#pragma unroll
                for (int m = 0; m < OWN; ++m) {
                    float *o = reinterpret_cast<float *>(&sh.sq[s + j * OWN + m][cl]);
                    *reinterpret_cast<float2 *>(o) = make_float2(sa[m], sb[m]);
                    o[2] = ys[m];
                }
            }
            __syncwarp();
        }
        gA[0] = add2(gA[0], tA[0]);
        gA[1] = add2(gA[1], tA[1]);
        __syncthreads();
        for (int i = threadIdx.x; i < TT * 2 * NP; i += kThreads) {
            const int row = i / (2 * NP), k = i % (2 * NP);
            float s = sh.bc[row][0][k];
#pragma unroll
            for (int q = 1; q < kBwdWarps; ++q)
                s += sh.bc[row][q][k];
            if (t0 + row < te)
                p.bc[(((t0 + row) * p.B + w.b) * p.grid.blocks + w.blk) * (2 * NP) + k] = s;
        }
#pragma unroll
        for (int r = 0; r < RP; ++r) {
            const int64_t t = t0 + pr + r * T::RG;
            const float4 s0 = sh.sq[pr + r * T::RG][pc], s1 = sh.sq[pr + r * T::RG][pc + 1];
            const float2 uv = unpack2<DT>(ru[r]);
            float2 raw = unpack2<DT>(rd[r]);
            raw.x += bias0;
            raw.y += bias1;
            float2 dy = unpack2<DT>(rg[r]);
            if (z) {
                const float2 zv = unpack2<DT>(rz[r]);
                const float sx = sigmoid(zv.x), sy = sigmoid(zv.y);
                const float2 gz = make_float2(dy.x * fmaf(D0, uv.x, s0.z) * sx * fmaf(zv.x, 1.f - sx, 1.f),
                                              dy.y * fmaf(D1, uv.y, s1.z) * sy * fmaf(zv.y, 1.f - sy, 1.f));
                if (p.gz && t < p.S)
                    store_pair<PAIRS>(p.gz + (t * p.B + w.b) * p.H + ch, t < te ? pack2<DT>(gz) : 0u, on0, on1);
                dy.x *= zv.x * sx;
                dy.y *= zv.y * sy;
            }
            float2 gr = make_float2(fmaf(uv.x, s0.y, s0.x), fmaf(uv.y, s1.y, s1.x));
            if (p.softplus) {
                gr.x *= raw.x > 20.f ? 1.f : sigmoid(raw.x);
                gr.y *= raw.y > 20.f ? 1.f : sigmoid(raw.y);
            }
            const float2 gu = make_float2(fmaf(s0.w, s0.y, D0 * dy.x), fmaf(s1.w, s1.y, D1 * dy.y));
            if (t < te) {
                gD = fma2(dy, uv, gD);
                gbias = add2(gbias, gr);
            }
            if (t < p.S) {
                const int64_t o = (t * p.B + w.b) * p.H + ch;
                store_pair<PAIRS>(p.gu + o, t < te ? pack2<DT>(gu) : 0u, on0, on1);
                store_pair<PAIRS>(p.gdelta + o, t < te ? pack2<DT>(gr) : 0u, on0, on1);
            }
        }
        __syncthreads();   // bc is written again in the next tile
    }
    if (live)
        *reinterpret_cast<float4 *>(p.ga + at * NP + n0) = make_float4(gA[0].x, gA[0].y, gA[1].x, gA[1].y);
    // grad_D and grad_delta_bias over the threads that share channels
    float4 *red = &sh.sq[0][0];
    __syncthreads();
    red[pr * T::CP + pc / 2] = make_float4(gD.x, gbias.x, gD.y, gbias.y);
    __syncthreads();
    if (pr == 0) {
        float4 s = red[pc / 2];
        for (int k = 1; k < T::RG; ++k) {
            const float4 v = red[k * T::CP + pc / 2];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        float2 *o = reinterpret_cast<float2 *>(p.gd) + (w.chunk * p.B + w.b) * p.H + ch;
        if (on0)
            o[0] = make_float2(s.x, s.y);
        if (on1)
            o[1] = make_float2(s.z, s.w);
    }
}

// grad_B and grad_C: the blocks of a group added up, one value per thread.
template <int DT>
__global__ void __launch_bounds__(256) mcc1d_ssm_scan_bwd_bc(const ScanParams p, int NP, uint16_t *gB, uint16_t *gC)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int k = (int)(i % (2 * NP)), n = k % NP;
    const int64_t q = i / (2 * NP), row = q / p.G, g = q - row * p.G;   // row = t B + b
    if (row >= p.S * p.B || n >= p.N)
        return;
    const int64_t t = row / p.B, b = row - t * p.B;
    float s = 0.f;
    if (t < clamped_length(p.lengths, b, p.S)) {
        const float *src = p.bc + (row * p.grid.blocks + g * p.grid.blocks_per_group) * (2 * NP) + k;
        for (int m = 0; m < p.grid.blocks_per_group; ++m)
            s += src[(int64_t)m * 2 * NP];
    }
    (k < NP ? gB : gC)[q * p.N + n] = (uint16_t)pack2<DT>(make_float2(s, 0.f));
}

// grad_A, grad_D and grad_delta_bias: the (chunk, sequence) parts of every
// column added up, 8 strided runs of parts and then the runs in order.
__global__ void __launch_bounds__(256) mcc1d_ssm_scan_bwd_sum(const ScanParams p, int NP, float *gA, float *gD, float *gbias)
{
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t i = (int64_t)blockIdx.x * 32 + lane, parts = p.chunks * p.B, acols = p.H * NP, cols = acols + 2 * p.H;
    float s = 0.f;
    if (i < cols) {
        const float *src = i < acols ? p.ga + i : p.gd + (i - acols);
        const int64_t step = i < acols ? acols : 2 * p.H;
        for (int64_t r = q; r < parts; r += 8)
            s += src[r * step];
    }
    red[q][lane] = s;
    __syncthreads();
    if (q != 0 || i >= cols)
        return;
#pragma unroll
    for (int k = 1; k < 8; ++k)
        s += red[k][lane];
    if (i < acols) {
        const int64_t h = i / NP;
        const int n = (int)(i - h * NP);
        if (n < p.N)
            gA[h * p.N + n] = s;
    } else {
        const int64_t c = i - acols;
        float *o = c & 1 ? gbias : gD;
        if (o)
            o[c / 2] = s;
    }
}

template <int DT, int NL, bool PAIRS>
int32_t run_pairs(const ScanParams &p, cudaStream_t s)
{
    constexpr int bytes = (int)sizeof(BwdShared<NL>);
    if (cudaFuncSetAttribute(mcc1d_ssm_scan_bwd<DT, NL, PAIRS>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
        cudaSuccess)
        return kErrCuda;
    mcc1d_ssm_scan_bwd<DT, NL, PAIRS><<<(unsigned)(p.grid.blocks * p.B * p.chunks), kThreads, bytes, s>>>(p);
    return cudaPeekAtLastError() == cudaSuccess ? kOk : kErrCuda;
}

template <int DT, int NL>
int32_t run(const ScanParams &p, cudaStream_t s)
{
    return p.pairs ? run_pairs<DT, NL, true>(p, s) : run_pairs<DT, NL, false>(p, s);
}

template <int DT>
int32_t run_nl(const ScanParams &p, int nl, cudaStream_t s)
{
    switch (nl) {
    case 1: return run<DT, 1>(p, s);
    case 2: return run<DT, 2>(p, s);
    case 4: return run<DT, 4>(p, s);
    case 8: return run<DT, 8>(p, s);
    default: return run<DT, 16>(p, s);
    }
}

}  // namespace

int32_t launch_scan_bwd_main(ScanParams p, const ScanPlan &pl, const mcc1d_scan_bwd_args &a, cudaStream_t s)
{
    p.grid = scan_grid(p.H, p.G, kThreads / pl.nl);
    const int32_t st = a.fwd.dtype == 0 ? run_nl<0>(p, pl.nl, s) : run_nl<1>(p, pl.nl, s);
    if (st != kOk)
        return st;
    const int64_t values = p.S * p.B * p.G * 2 * pl.np;
    const unsigned grid = (unsigned)((values + 255) / 256);
    if (a.fwd.dtype == 0)
        mcc1d_ssm_scan_bwd_bc<0><<<grid, 256, 0, s>>>(p, pl.np, (uint16_t *)a.grad_B, (uint16_t *)a.grad_C);
    else
        mcc1d_ssm_scan_bwd_bc<1><<<grid, 256, 0, s>>>(p, pl.np, (uint16_t *)a.grad_B, (uint16_t *)a.grad_C);
    const int64_t cols = p.H * (pl.np + 2);
    mcc1d_ssm_scan_bwd_sum<<<(unsigned)((cols + 31) / 32), 256, 0, s>>>(p, pl.np, a.grad_A, a.grad_D, a.grad_delta_bias);
    return cudaPeekAtLastError() == cudaSuccess ? kOk : kErrCuda;
}

}  // namespace mcc1d
