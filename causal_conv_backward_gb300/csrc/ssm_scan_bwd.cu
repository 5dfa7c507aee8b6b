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
//
// 14 bytes per (token, channel) have to move, and about 21 N flops with 3 N
// exponentials (the states are run through three times) are computed: it is
// bound by instructions, about 38 per 128 (channel, state) steps in the first
// pass and 114 in this one, of which 63 are the run back (16 of them its sums
// over a channel's lanes, 7 those over a warp's channels) and 9 the run
// forward. Four blocks of 128 registers per SM beat three of 168 (4096 x 8 x
// 2048: 1608 against 1632 us), which is why the tile's rows are read again at
// its end and the warps' sums take the place of the states they have used.
// bf16, N = 16: 813 us on 2048 x 8 x 2048, 3095 on 1024 x 32 x 4096; N = 4, 8
// and 32 on 2048 x 8 x 2048: 445, 539 and 1491.
#include "plan.h"
#include "ssm_scan.cuh"

namespace mcc1d {

namespace {

constexpr int kSub = 2;          // rows whose states and decays sit in registers
constexpr int kBlocksPerSM = 4;

template <int NL>
struct BwdShared {
    using T = BwdMainTile<NL>;
    static constexpr int TT = T::TT;
    // dt, dt u, dy, dt; the first three then sum A log2e q, sum g B, y. A lane's channels lie in planes of their
    // own, so that the lanes of a warp read neighbouring 16 bytes.
    float4 sq[TT][T::K][T::CB / T::K];
    float4 hs[TT / kSub][T::K][T::EL_THREADS];       // states before each run of kSub rows
    float sB[TT][T::NP], sC[TT][T::NP];
    // A warp's grad_B and grad_C of row s + i take the place of its own hs[s / kSub][i], which it has read by then.
    static_assert(kSub <= T::K && 2 * T::NP <= 4 * 32, "a row of sums fits a warp's states of one channel");
    static_assert(kSub == 2, "an odd number of rows leaves one free in the last run");
    __device__ __forceinline__ float *bc(int row, int warp)
    {
        return reinterpret_cast<float *>(&hs[row / kSub][row % kSub][32 * warp]);
    }
    // An odd number of rows leaves the last run a row that is no token. It must not follow the last token: with dt
    // = 0 it would add nothing to grad_A but 0 times the final state, which may be infinite where no token's grad_A
    // is. So it goes before it (clear_last, the last token moves up; its results move back with fetch_last). A test
    // in the walk back costs every tile of N = 8 7 % and of N = 32 and 64 3 to 4 %, this nothing but in such tiles.
    __device__ __forceinline__ void clear_last(int rows)
    {
        for (int i = threadIdx.x; i < T::CB; i += T::EL_THREADS) {
            (&sq[rows][0][0])[i] = (&sq[rows - 1][0][0])[i];
            (&sq[rows - 1][0][0])[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int i = threadIdx.x; i < T::NP; i += T::EL_THREADS) {
            sB[rows][i] = sB[rows - 1][i];
            sC[rows][i] = sC[rows - 1][i];
            sB[rows - 1][i] = sC[rows - 1][i] = 0.f;
        }
        __syncthreads();
    }
    __device__ __forceinline__ void fetch_last(int rows)
    {
        for (int i = threadIdx.x; i < T::CB; i += T::EL_THREADS)
            (&sq[rows - 1][0][0])[i] = (&sq[rows][0][0])[i];
        for (int i = threadIdx.x; i < 2 * T::NP * T::WARPS; i += T::EL_THREADS)
            bc(rows - 1, i / (2 * T::NP))[i % (2 * T::NP)] = bc(rows, i / (2 * T::NP))[i % (2 * T::NP)];
        __syncthreads();
    }
};

template <int DT, int NL, bool PAIRS>
__global__ void __launch_bounds__(BwdMainTile<NL>::EL_THREADS, kBlocksPerSM) mcc1d_ssm_scan_bwd(const ScanParams p)
{
    using T = BwdMainTile<NL>;
    using Sh = BwdShared<NL>;
    constexpr int NP = T::NP, CL = T::CL, TT = T::TT, RG = T::RG, RP = T::RP, K = T::K;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Sh &sh = *reinterpret_cast<Sh *>(raw_shared);

    next_may_start();
    previous_done();
    const ScanWhere w = scan_where<T>(p);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = T::state_lane(lane), n0 = 4 * j, ci = T::channel_lane(lane);
    const int cw = warp * CL + ci, cl = cw * K;
    const int64_t te = clamped_length(p.lengths, w.b, p.S);
    const int pc = 2 * (threadIdx.x % T::CP), pr = threadIdx.x / T::CP;
    const bool on0 = pc < w.nc, on1 = pc + 1 < w.nc;
    const int64_t ch = w.c0 + (on0 ? pc : 0);
    const uint16_t *Bm = p.Bm + w.b * p.Bb + w.g * p.Bg, *Cm = p.Cm + w.b * p.Cb + w.g * p.Cg;
    float2 bias = make_float2(0.f, 0.f), D = make_float2(0.f, 0.f);
    if (p.dbias)
        bias = make_float2(on0 ? p.dbias[ch] : 0.f, on1 ? p.dbias[ch + 1] : 0.f);
    if (p.D)
        D = make_float2(on0 ? p.D[ch] : 0.f, on1 ? p.D[ch + 1] : 0.f);

    float2 A2[K][2], X[K][2], gA[K][2];
    int64_t hc[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const bool there = cl + k < w.nc;
        hc[k] = w.b * p.H + w.c0 + (there ? cl + k : 0);
        // A lane past the group's channels holds zeros: its steps are softplus(0), under which another channel's
        // growing state or gradient would pass fp32, and infinity times its zero input is NaN in the group's sums.
        const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = there ? load_states(p.A + (hc[k] - w.b * p.H) * p.N, n0, p.N, p.vecA) : none;
        A2[k][0] = make_float2(a.x * kLog2e, a.y * kLog2e);
        A2[k][1] = make_float2(a.z * kLog2e, a.w * kLog2e);
        const float4 x = there ? *reinterpret_cast<const float4 *>(p.r + (w.chunk * p.B * p.H + hc[k]) * NP + n0) : none;
        X[k][0] = make_float2(x.x, x.y);
        X[k][1] = make_float2(x.z, x.w);
        gA[k][0] = gA[k][1] = make_float2(0.f, 0.f);
    }
    float2 gD = make_float2(0.f, 0.f), gbias = make_float2(0.f, 0.f);

    const int64_t tile0 = w.chunk * p.tiles_per_chunk;
    const int64_t tile1 = tile0 + p.tiles_per_chunk < p.tiles ? tile0 + p.tiles_per_chunk : p.tiles;
    const int64_t live_end = (te + TT - 1) / TT < tile1 ? (te + TT - 1) / TT : tile1;   // past the tiles with tokens
    const int64_t os = RG * p.B * p.H;
    // past the sequence's end: zeros
    for (int64_t tile = tile1 - 1; tile >= tile0 && tile >= live_end; --tile) {
        int64_t o = ((tile * TT + pr) * p.B + w.b) * p.H + ch;
#pragma unroll
        for (int r = 0; r < RP; ++r, o += os)
            if (tile * TT + pr + r * RG < p.S) {
                store_pair<PAIRS>(p.gu + o, 0u, on0, on1);
                store_pair<PAIRS>(p.gdelta + o, 0u, on0, on1);
                if (p.gz)
                    store_pair<PAIRS>(p.gz + o, 0u, on0, on1);
            }
    }
    auto load = [&](int64_t tile, uint32_t (&ru)[RP], uint32_t (&rd)[RP], uint32_t (&rz)[RP], uint32_t (&rg)[RP]) {
        const int64_t trow = tile * TT + pr;
        const int rows = (int)(te - tile * TT < TT ? te - tile * TT : TT);
        const uint16_t *u = p.u + w.b * p.ub + ch + trow * p.us, *delta = p.delta + w.b * p.db + ch + trow * p.ds;
        const uint16_t *z = p.z ? p.z + w.b * p.zb + ch + trow * p.zs : nullptr, *gy = p.gy + w.b * p.gb + ch + trow * p.gs;
#pragma unroll
        for (int r = 0; r < RP; ++r) {
            const bool ok = pr + r * RG < rows;
            ru[r] = load_pair<PAIRS>(u, ok && on0, ok && on1);
            rd[r] = load_pair<PAIRS>(delta, ok && on0, ok && on1);
            rg[r] = load_pair<PAIRS>(gy, ok && on0, ok && on1);
            u += RG * p.us;
            delta += RG * p.ds;
            gy += RG * p.gs;
            if (p.z) {
                rz[r] = load_pair<PAIRS>(z, ok && on0, ok && on1);
                z += RG * p.zs;
            }
        }
    };
    // a thread's sums of grad_B and grad_C in the tile: column bk of rows brow, brow + BR, ..
    constexpr int BR = T::EL_THREADS / (2 * NP), BN = TT > BR ? TT / BR : 1;
    static_assert(BR >= 1 && (TT % BR == 0 || BR > TT), "a tile is whole passes");
    const int bk = threadIdx.x % (2 * NP), brow = threadIdx.x / (2 * NP);
    const int64_t bstep = (int64_t)p.B * p.grid.blocks * (2 * NP);
    BcTile<T, true> bc;
    bc.start(p, Bm + (live_end - 1) * TT * p.Bs, Cm + (live_end - 1) * TT * p.Cs, threadIdx.x, -1);
    for (int64_t tile = live_end - 1; tile >= tile0; --tile) {
        const int64_t t0 = tile * TT;
        const int rows = (int)(te - t0 < TT ? te - t0 : TT), all = (int)(p.S - t0 < TT ? p.S - t0 : TT);
        uint32_t ru[RP], rd[RP], rz[RP], rg[RP];   // read again at the tile's end rather than held
        load(tile, ru, rd, rz, rg);
        bc.load(p, rows);
        bc.template put<DT>(p, sh.sB, sh.sC);
        {
            // branches that are the same for every row stand outside the loops over rows
            float2 dt[RP], g[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                dt[r] = add2(unpack2<DT>(rd[r]), bias);
                g[r] = unpack2<DT>(rg[r]);
            }
            if (p.softplus) {
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    dt[r] = softplus2(dt[r]);
            }
            if (p.z) {
#pragma unroll
                for (int r = 0; r < RP; ++r) {
                    const float2 zv = unpack2<DT>(rz[r]);
                    g[r] = mul2(g[r], mul2(zv, sigmoid2(zv)));
                }
            }
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                const int row = pr + r * RG;
                if (row >= rows)
                    dt[r] = make_float2(0.f, 0.f);
                const float2 du = mul2(dt[r], unpack2<DT>(ru[r]));
                sh.sq[row][0][pc / 2] = make_float4(dt[r].x, du.x, g[r].x, dt[r].x);
                sh.sq[row][1][pc / 2] = make_float4(dt[r].y, du.y, g[r].y, dt[r].y);
            }
        }
        // the state at the tile's start: from the chunk's zero start, and what entered the chunk
        float2 h[K][2];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t ct = tile * p.B * p.H + hc[k];
            const float4 s = *reinterpret_cast<const float4 *>(p.cp + ct * NP + n0);
            const float4 e = *reinterpret_cast<const float4 *>(p.e + (w.chunk * p.B * p.H + hc[k]) * NP + n0);
            const float d = p.cpdt[ct];
            h[k][0] = grown(make_float2(e.x, e.y), d, A2[k][0], make_float2(s.x, s.y));
            h[k][1] = grown(make_float2(e.z, e.w), d, A2[k][1], make_float2(s.z, s.w));
        }
        __syncthreads();
        if (rows & 1)
            sh.clear_last(rows);
#pragma unroll 1
        for (int s = 0; s < TT; s += kSub) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                sh.hs[s / kSub][k][threadIdx.x] = make_float4(h[k][0].x, h[k][0].y, h[k][1].x, h[k][1].y);
            if (s + kSub == TT)
                break;
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const float4 bv = *reinterpret_cast<const float4 *>(&sh.sB[s + i][n0]);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float2 dd = *reinterpret_cast<const float2 *>(&sh.sq[s + i][k][cw]);
                    const float2 dt2 = make_float2(dd.x, dd.x), du2 = make_float2(dd.y, dd.y);
                    h[k][0] = fma2(decay2(dt2, A2[k][0]), h[k][0], mul2(du2, make_float2(bv.x, bv.y)));
                    h[k][1] = fma2(decay2(dt2, A2[k][1]), h[k][1], mul2(du2, make_float2(bv.z, bv.w)));
                }
            }
        }
        float2 tA[K][2];   // the tile's part of grad_A: short sums first
#pragma unroll
        for (int k = 0; k < K; ++k)
            tA[k][0] = tA[k][1] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int s = (rows - 1) / kSub * kSub; s >= 0; s -= kSub) {   // from the run of the last token
            float2 hh[kSub + 1][K][2], aa[kSub][K][2];
            float ys[K * kSub], sa[K * kSub], sb[K * kSub];     // of (step, channel)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float4 v = sh.hs[s / kSub][k][threadIdx.x];
                hh[0][k][0] = make_float2(v.x, v.y);
                hh[0][k][1] = make_float2(v.z, v.w);
            }
            __syncwarp();   // the warp's sums take the place of these
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const float4 bv = *reinterpret_cast<const float4 *>(&sh.sB[s + i][n0]);
                const float4 cv = *reinterpret_cast<const float4 *>(&sh.sC[s + i][n0]);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float2 dd = *reinterpret_cast<const float2 *>(&sh.sq[s + i][k][cw]);
                    const float2 dt2 = make_float2(dd.x, dd.x), du2 = make_float2(dd.y, dd.y);
                    aa[i][k][0] = decay2(dt2, A2[k][0]);
                    aa[i][k][1] = decay2(dt2, A2[k][1]);
                    hh[i + 1][k][0] = fma2(aa[i][k][0], hh[i][k][0], mul2(du2, make_float2(bv.x, bv.y)));
                    hh[i + 1][k][1] = fma2(aa[i][k][1], hh[i][k][1], mul2(du2, make_float2(bv.z, bv.w)));
                    const float2 y = fma2(hh[i + 1][k][0], make_float2(cv.x, cv.y),
                                          mul2(hh[i + 1][k][1], make_float2(cv.z, cv.w)));
                    ys[i * K + k] = y.x + y.y;
                }
            }
#pragma unroll
            for (int i = kSub - 1; i >= 0; --i) {
                const float4 bv = *reinterpret_cast<const float4 *>(&sh.sB[s + i][n0]);
                const float4 cv = *reinterpret_cast<const float4 *>(&sh.sC[s + i][n0]);
                float2 v0, v1, c0, c1;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float4 dd = sh.sq[s + i][k][cw];
                    const float2 dt2 = make_float2(dd.x, dd.x), du2 = make_float2(dd.y, dd.y), dy2 = make_float2(dd.z, dd.z);
                    const float2 g0 = fma2(dy2, make_float2(cv.x, cv.y), X[k][0]);
                    const float2 g1 = fma2(dy2, make_float2(cv.z, cv.w), X[k][1]);
                    const float2 b2 = fma2(g0, make_float2(bv.x, bv.y), mul2(g1, make_float2(bv.z, bv.w)));
                    sb[i * K + k] = b2.x + b2.y;
                    X[k][0] = mul2(aa[i][k][0], g0);
                    X[k][1] = mul2(aa[i][k][1], g1);
                    const float2 q0 = mul2(X[k][0], hh[i][k][0]), q1 = mul2(X[k][1], hh[i][k][1]);
                    const float2 a2 = fma2(A2[k][0], q0, mul2(A2[k][1], q1));
                    sa[i * K + k] = a2.x + a2.y;
                    tA[k][0] = fma2(dt2, q0, tA[k][0]);
                    tA[k][1] = fma2(dt2, q1, tA[k][1]);
                    v0 = k == 0 ? mul2(g0, du2) : fma2(g0, du2, v0);
                    v1 = k == 0 ? mul2(g1, du2) : fma2(g1, du2, v1);
                    c0 = k == 0 ? mul2(hh[i + 1][k][0], dy2) : fma2(hh[i + 1][k][0], dy2, c0);
                    c1 = k == 0 ? mul2(hh[i + 1][k][1], dy2) : fma2(hh[i + 1][k][1], dy2, c1);
                }
                float v[8] = {v0.x, v0.y, v1.x, v1.y, c0.x, c0.y, c1.x, c1.y};
                lanes_sum<8, CL, NL == 1 ? 1 : 2, NL == 1 ? 1 : 2>(v, lane);
                constexpr int KEEP = CL >= 8 ? 1 : 8 / CL;
                if (ci < 8) {
                    const int k = (ci * KEEP) % 8;      // v[0..KEEP-1] are values k.. of the eight
                    float *o = sh.bc(s + i, warp) + (k / 4) * NP + n0 + k % 4;
#pragma unroll
                    for (int m = 0; m < KEEP; ++m)
                        o[m] = v[m];
                }
            }
            constexpr int N = K * kSub, OWN = NL >= N ? 1 : N / NL;
            lanes_sum<N, NL, 1, CL>(ys, lane);
            lanes_sum<N, NL, 1, CL>(sa, lane);
            lanes_sum<N, NL, 1, CL>(sb, lane);
            if (j < N) {
#pragma unroll
                for (int m = 0; m < OWN; ++m) {
                    const int q = j * OWN + m;          // (step, channel)
                    float *o = reinterpret_cast<float *>(&sh.sq[s + q / K][q % K][cw]);
                    *reinterpret_cast<float2 *>(o) = make_float2(sa[m], sb[m]);
                    o[2] = ys[m];
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            gA[k][0] = add2(gA[k][0], tA[k][0]);
            gA[k][1] = add2(gA[k][1], tA[k][1]);
        }
        __syncthreads();
        if (rows & 1)
            sh.fetch_last(rows);
        load(tile, ru, rd, rz, rg);
        float *to = p.bc + (t0 + brow) * bstep + (w.b * p.grid.blocks + w.blk) * (2 * NP) + bk;
#pragma unroll
        for (int i = 0; i < BN; ++i, to += BR * bstep) {
            const int row = brow + i * BR;
            if (row >= rows)
                break;
            float s = sh.bc(row, 0)[bk];
#pragma unroll
            for (int q = 1; q < T::WARPS; ++q)
                s += sh.bc(row, q)[bk];
            *to = s;
        }
        const int64_t o = ((t0 + pr) * p.B + w.b) * p.H + ch;
        const float2 one = make_float2(1.f, 1.f);
        float2 dy[RP], slope[RP];
#pragma unroll
        for (int r = 0; r < RP; ++r) {
            dy[r] = unpack2<DT>(rg[r]);
            slope[r] = one;
        }
        if (p.z) {
            uint32_t gz[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                const int row = pr + r * RG;
                const float2 y = make_float2(sh.sq[row][0][pc / 2].z, sh.sq[row][1][pc / 2].z);
                const float2 zv = unpack2<DT>(rz[r]), sz = sigmoid2(zv);
                // d/dz [z sz] = sz (1 + z (1 - sz))
                const float2 d = mul2(sz, fma2(zv, make_float2(1.f - sz.x, 1.f - sz.y), one));
                gz[r] = pack2<DT>(mul2(mul2(dy[r], fma2(D, unpack2<DT>(ru[r]), y)), d));
                dy[r] = mul2(dy[r], mul2(zv, sz));
            }
            if (p.gz) {
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    if (pr + r * RG < all)
                        store_pair<PAIRS>(p.gz + o + r * os, pr + r * RG < rows ? gz[r] : 0u, on0, on1);
            }
        }
        if (p.softplus) {
#pragma unroll
            for (int r = 0; r < RP; ++r)
                slope[r] = sigmoid2(add2(unpack2<DT>(rd[r]), bias));
        }
#pragma unroll
        for (int r = 0; r < RP; ++r) {
            const int row = pr + r * RG;
            const float4 s0 = sh.sq[row][0][pc / 2], s1 = sh.sq[row][1][pc / 2];
            const float2 uv = unpack2<DT>(ru[r]), sb = make_float2(s0.y, s1.y);
            constexpr float ln2 = 0.693147181f;
            float2 gr = mul2(fma2(uv, sb, mul2(make_float2(s0.x, s1.x), make_float2(ln2, ln2))), slope[r]);
            float2 gu = fma2(make_float2(s0.w, s1.w), sb, mul2(D, dy[r]));
            if (row >= rows)
                gr = gu = make_float2(0.f, 0.f);
            gD = fma2(dy[r], uv, gD);      // past the end both are zeros
            gbias = add2(gbias, gr);
            if (row < all) {
                store_pair<PAIRS>(p.gu + o + r * os, pack2<DT>(gu), on0, on1);
                store_pair<PAIRS>(p.gdelta + o + r * os, pack2<DT>(gr), on0, on1);
            }
        }
        __syncthreads();   // hs is written again in the next tile
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (cl + k < w.nc)
            *reinterpret_cast<float4 *>(p.ga + (w.chunk * p.B * p.H + hc[k]) * NP + n0) =
                make_float4(gA[k][0].x, gA[k][0].y, gA[k][1].x, gA[k][1].y);
    // grad_D and grad_delta_bias over the threads that share channels
    float4 *red = &sh.sq[0][0][0];
    __syncthreads();
    red[pr * T::CP + pc / 2] = make_float4(gD.x, gbias.x, gD.y, gbias.y);
    __syncthreads();
    if (pr == 0) {
        float4 s = red[pc / 2];
        for (int k = 1; k < RG; ++k) {
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

// What is left to add up, in one launch. The first bc_blocks blocks: grad_B and
// grad_C, the blocks of a group, one value per thread. The others: grad_A,
// grad_D and grad_delta_bias, the (chunk, sequence) parts of every column, 8
// strided runs of parts and then the runs in order.
template <int DT>
__global__ void __launch_bounds__(256) mcc1d_ssm_scan_bwd_sums(const ScanParams p, int NP, unsigned bc_blocks, uint16_t *gB,
                                                              uint16_t *gC, float *gA, float *gD, float *gbias)
{
    previous_done();
    if (blockIdx.x < bc_blocks) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        const int k = (int)(i % (2 * NP)), n = k % NP;
        const int64_t q = i / (2 * NP), row = q / p.G, g = q - row * p.G;   // row = t B + b
        if (row >= p.S * p.B || n >= p.N)
            return;
        const int64_t t = row / p.B, b = row - t * p.B;
        float s = 0.f;
        if (t < clamped_length(p.lengths, b, p.S)) {
            const float *src = p.bc + (row * p.grid.blocks + g * p.grid.blocks_per_group) * (2 * NP) + k;
#pragma unroll 8
            for (int m = 0; m < p.grid.blocks_per_group; ++m)
                s += src[(int64_t)m * 2 * NP];
        }
        (k < NP ? gB : gC)[q * p.N + n] = (uint16_t)pack2<DT>(make_float2(s, 0.f));
        return;
    }
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t i = (int64_t)(blockIdx.x - bc_blocks) * 32 + lane, parts = p.chunks * p.B, acols = p.H * NP, cols = acols + 2 * p.H;
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
    static SharedReady ready;
    if (!ready.set((const void *)mcc1d_ssm_scan_bwd<DT, NL, PAIRS>, bytes))
        return kErrCuda;
    return launch_as(true, mcc1d_ssm_scan_bwd<DT, NL, PAIRS>, scan_launch_grid(p), BwdMainTile<NL>::EL_THREADS, bytes, s, p);
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

int32_t launch_scan_bwd_main(const ScanParams &p, const ScanPlan &pl, const mcc1d_scan_bwd_args &a, cudaStream_t s)
{
    const int32_t st = a.fwd.dtype == 0 ? run_nl<0>(p, pl.nl, s) : run_nl<1>(p, pl.nl, s);
    if (st != kOk)
        return st;
    const int64_t values = p.S * p.B * p.G * 2 * pl.np, cols = p.H * (pl.np + 2);
    const unsigned bc_blocks = (unsigned)((values + 255) / 256), grid = bc_blocks + (unsigned)((cols + 31) / 32);
    const auto sums = a.fwd.dtype == 0 ? mcc1d_ssm_scan_bwd_sums<0> : mcc1d_ssm_scan_bwd_sums<1>;
    return launch_as(true, sums, grid, 256, 0, s, p, pl.np, bc_blocks, (uint16_t *)a.grad_B, (uint16_t *)a.grad_C, a.grad_A, a.grad_D,
                  a.grad_delta_bias);
}

}  // namespace mcc1d
