// ssm_scan.cu - the selective scan over prompts and for single tokens.
//
//   h(t)[n] = exp(dt A[n]) h(t-1)[n] + dt u B(t)[n],  y(t) = (C(t).h(t) + D u) z sigmoid(z)
//
// The call moves 8 bytes per (token, channel) and computes, for each of its N
// states, one exponential and four multiply-adds. At N = 16 that is more than
// memory: a scheduler issues a warp's exponential in 4 cycles and a packed
// multiply-add in 2 (measured), so 128 (channel, state) steps take 16 cycles
// of each pipe where their bytes take 9, and about 17 instructions besides
// what each element needs once (loads, softplus, gate: some 40 per element).
// The design therefore spends as few other instructions per state as it can.
// A channel's states sit four to a lane (ssm_scan.cuh): enough warps for a few
// thousand channels without cutting the sequence. Measured, bf16, N = 16:
// 690 us on 1024 x 32 x 4096 (48 cycles per 128 steps, issuing on 64 % of
// cycles), 418 us on 4096 x 8 x 2048 (512 blocks on 152 SMs: four on some and
// three on others), 463 us on 131072 x 1 x 384 (cut in chunks).
//
// Where sequences and channels are too few to fill the machine the time axis
// is cut into chunks: each chunk's state from a zero start and its sum of dt
// (which fixes its decay exp(A sum dt)) are computed, the chunks are joined in
// order, and the outputs are computed chunk by chunk from the joined states.
#include <algorithm>

#include "plan.h"
#include "ssm_scan.cuh"

namespace mcc1d {

namespace {

// What a pass leaves behind: outputs; a chunk's end state; or, for the
// backward, also the states at tile starts and the gradient that reaches the
// chunk's start from the outputs inside it.
enum { kOutputs = 0, kSummary = 1, kSummaryGrad = 2 };

template <class T, int MODE>
struct ScanShared {
    static constexpr bool kY = MODE == kOutputs, kR = MODE == kSummaryGrad, kC = kY || kR;
    static constexpr int NL = T::NL, TT = T::TT, CB = T::CB;
    // a lane's row of y: CL mod 32, so that the lanes of a warp are on 32 different banks
    static constexpr int YS = CB + (T::CL * T::K + 32 * T::WARPS - CB % 32) % 32;
    float2 sd[2][TT][CB];                    // dt, dt u
    float sB[2][TT][T::NP];
    float sC[2][kC ? TT : 1][T::NP];
    float sy[2][kY ? TT : 1][NL][YS];        // a lane's part of y
    float sg[2][kR ? TT : 1][CB];            // the gradient of y
    uint2 raw[2][kY ? T::RP : 1][T::EL_THREADS];   // u and z of a tile, until its outputs are due
};

// Every thread of the block, from either role's code.
__device__ __forceinline__ void block_barrier(int threads) { asm volatile("bar.sync 0, %0;" ::"r"(threads) : "memory"); }

template <class T, int DT, int MODE, bool PAIRS>
__global__ void __launch_bounds__(T::THREADS, MODE == kSummaryGrad ? 3 : 4) mcc1d_ssm_scan(const ScanParams p)
{
    using Sh = ScanShared<T, MODE>;
    constexpr int NP = T::NP, NL = T::NL, TT = T::TT, RG = T::RG, RP = T::RP, K = T::K;
    constexpr bool kY = Sh::kY, kR = Sh::kR, kC = Sh::kC;
    constexpr int U = 2;                     // steps of the recurrence taken together
    extern __shared__ __align__(16) unsigned char raw_shared[];
    Sh &sh = *reinterpret_cast<Sh *>(raw_shared);

    // outputs after a join read its states; the passes before a join let it be set up
    if (kY)
        previous_done();
    else
        next_may_start();
    const ScanWhere w = scan_where<T>(p);
    const int64_t te = clamped_length(p.lengths, w.b, p.S);
    const int64_t tile0 = w.chunk * p.tiles_per_chunk;
    const int64_t tile1 = tile0 + p.tiles_per_chunk < p.tiles ? tile0 + p.tiles_per_chunk : p.tiles;
    // the chunk's tiles that hold tokens, and the rows of its i-th tile that do; all but the last are full
    const int64_t live_end = (te + TT - 1) / TT < tile1 ? (te + TT - 1) / TT : tile1;
    const int n_tiles = live_end > tile0 ? (int)(live_end - tile0) : 0;
    const int last_rows = n_tiles > 0 ? (int)(te - (tile0 + n_tiles - 1) * TT < TT ? te - (tile0 + n_tiles - 1) * TT : TT) : 0;
    auto rows_in = [&](int i) { return i < n_tiles - 1 ? TT : last_rows; };
    const int warp = threadIdx.x >> 5;

    if (warp >= T::WARPS) {
        const int id = threadIdx.x - 32 * T::WARPS;
        const int pc = 2 * (id % T::CP), pr = id / T::CP;
        const bool on0 = pc < w.nc, on1 = pc + 1 < w.nc;
        const int64_t ch = w.c0 + (on0 ? pc : 0), trow = tile0 * TT + pr;
        const uint16_t *u = p.u + w.b * p.ub + ch + trow * p.us, *delta = p.delta + w.b * p.db + ch + trow * p.ds;
        const uint16_t *z = kC && p.z ? p.z + w.b * p.zb + ch + trow * p.zs : nullptr;
        const uint16_t *gy = kR ? p.gy + w.b * p.gb + ch + trow * p.gs : nullptr;
        uint16_t *y = kY ? p.y + (trow * p.B + w.b) * p.H + ch : nullptr;
        const int64_t ys = RG * p.B * p.H;
        const int64_t us = RG * p.us, ds = RG * p.ds, zs = RG * p.zs, gs = RG * p.gs;
        float2 bias = make_float2(0.f, 0.f), D = make_float2(0.f, 0.f);
        if (p.dbias)
            bias = make_float2(on0 ? p.dbias[ch] : 0.f, on1 ? p.dbias[ch + 1] : 0.f);
        if (kY && p.D)
            D = make_float2(on0 ? p.D[ch] : 0.f, on1 ? p.D[ch + 1] : 0.f);

        uint32_t ru[RP], rd[RP], rz[RP], rg[RP];
        BcTile<T, kC> bc;
        bc.start(p, p.Bm + w.b * p.Bb + w.g * p.Bg + tile0 * TT * p.Bs, p.Cm + w.b * p.Cb + w.g * p.Cg + tile0 * TT * p.Cs, id, 1);
        // Branches that are the same for every row stand outside the loops over rows, whose bodies interleave.
        auto load = [&](int rows) {
            bool ok[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                ok[r] = pr + r * RG < rows;
                ru[r] = load_pair<PAIRS>(u, ok[r] && on0, ok[r] && on1);
                rd[r] = load_pair<PAIRS>(delta, ok[r] && on0, ok[r] && on1);
                rz[r] = 0u;
                u += us;
                delta += ds;
                if (kR) {
                    rg[r] = load_pair<PAIRS>(gy, ok[r] && on0, ok[r] && on1);
                    gy += gs;
                }
            }
            if (kC && p.z) {
#pragma unroll
                for (int r = 0; r < RP; ++r, z += zs)
                    rz[r] = load_pair<PAIRS>(z, ok[r] && on0, ok[r] && on1);
            }
            bc.load(p, rows);
        };
        // what the recurrence needs of tile i, whose rows are in registers; then the next tile's are asked for
        auto before = [&](int i) {
            const int buf = i & 1, rows = rows_in(i);
            float2 dt[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r)
                dt[r] = add2(unpack2<DT>(rd[r]), bias);
            if (p.softplus) {
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    dt[r] = softplus2(dt[r]);
            }
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                const int row = pr + r * RG;
                if (row >= rows)
                    dt[r] = make_float2(0.f, 0.f);
                const float2 du = mul2(dt[r], unpack2<DT>(ru[r]));
                *reinterpret_cast<float4 *>(&sh.sd[buf][row][pc]) = make_float4(dt[r].x, du.x, dt[r].y, du.y);
                if (kY)
                    sh.raw[buf][r][id] = make_uint2(ru[r], rz[r]);
            }
            if (kR) {
                float2 g[RP];
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    g[r] = unpack2<DT>(rg[r]);
                if (p.z) {
#pragma unroll
                    for (int r = 0; r < RP; ++r) {
                        const float2 zv = unpack2<DT>(rz[r]);
                        g[r] = mul2(g[r], mul2(zv, sigmoid2(zv)));
                    }
                }
#pragma unroll
                for (int r = 0; r < RP; ++r)
                    *reinterpret_cast<float2 *>(&sh.sg[buf][pr + r * RG][pc]) = g[r];
            }
            bc.template put<DT>(p, sh.sB[buf], sh.sC[buf]);
            if (i + 1 < n_tiles)
                load(rows_in(i + 1));
        };
        // the outputs of tile i
        const int last_all = (int)(p.S - (live_end - 1) * TT < TT ? p.S - (live_end - 1) * TT : TT);
        auto after = [&](int i) {
            const int buf = i & 1, rows = rows_in(i), all = i < n_tiles - 1 ? TT : last_all;
            float2 v[RP];
            uint2 rv[RP];
#pragma unroll
            for (int r = 0; r < RP; ++r) {
                const int row = pr + r * RG;
                rv[r] = sh.raw[buf][r][id];
                v[r] = *reinterpret_cast<const float2 *>(&sh.sy[buf][row][0][pc]);
#pragma unroll
                for (int k = 1; k < NL; ++k)
                    v[r] = add2(v[r], *reinterpret_cast<const float2 *>(&sh.sy[buf][row][k][pc]));
                v[r] = fma2(D, unpack2<DT>(rv[r].x), v[r]);
            }
            if (p.z) {
#pragma unroll
                for (int r = 0; r < RP; ++r) {
                    const float2 zv = unpack2<DT>(rv[r].y);
                    v[r] = mul2(v[r], mul2(zv, sigmoid2(zv)));
                }
            }
#pragma unroll
            for (int r = 0; r < RP; ++r, y += ys) {
                const int row = pr + r * RG;
                if (row < all)
                    store_pair<PAIRS>(y, row < rows ? pack2<DT>(v[r]) : 0u, on0, on1);
            }
        };
        if (n_tiles > 0) {
            load(rows_in(0));
            before(0);
        }
        block_barrier(T::THREADS);
        for (int i = 0; i < n_tiles; ++i) {
            if (kY && i > 0)
                after(i - 1);
            if (i + 1 < n_tiles)
                before(i + 1);
            block_barrier(T::THREADS);
        }
        if (kY) {
            if (n_tiles > 0)
                after(n_tiles - 1);
            // past the sequence's end: zeros, and the state stays
            for (int64_t tile = tile0 + n_tiles; tile < tile1; ++tile) {
                const int all = (int)(p.S - tile * TT < TT ? p.S - tile * TT : TT);
#pragma unroll
                for (int r = 0; r < RP; ++r, y += ys)
                    if (pr + r * RG < all)
                        store_pair<PAIRS>(y, 0u, on0, on1);
            }
        }
        return;
    }

    // the recurrence: a lane's four states of each of its channels
    const int lane = threadIdx.x & 31, j = T::state_lane(lane), n0 = 4 * j;
    const int cl = (warp * T::CL + T::channel_lane(lane)) * K;   // first channel, within the block
    float2 A2[K][2], h[K][2], q[K][2], R[K][2];
    float dtsum[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t hc = w.c0 + (cl + k < w.nc ? cl + k : 0);
        const float4 a = load_states(p.A + hc * p.N, n0, p.N, p.vecA);
        A2[k][0] = make_float2(a.x * kLog2e, a.y * kLog2e);
        A2[k][1] = make_float2(a.z * kLog2e, a.w * kLog2e);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (kY) {
            if (p.chunks > 1)
                s = *reinterpret_cast<const float4 *>(p.e + ((w.chunk * p.B + w.b) * p.H + hc) * NP + n0);
            else if (p.h0)
                s = load_states(p.h0 + (w.b * p.H + hc) * p.N, n0, p.N, p.vecState);
        }
        h[k][0] = make_float2(s.x, s.y);
        h[k][1] = make_float2(s.z, s.w);
        q[k][0] = q[k][1] = make_float2(1.f, 1.f);
        R[k][0] = R[k][1] = make_float2(0.f, 0.f);
        dtsum[k] = 0.f;
    }
    block_barrier(T::THREADS);
    for (int tile = 0; tile < n_tiles; ++tile) {
        const int buf = tile & 1;
        if (kR) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (cl + k < w.nc) {
                    const int64_t at = ((tile0 + tile) * p.B + w.b) * p.H + w.c0 + cl + k;
                    *reinterpret_cast<float4 *>(p.cp + at * NP + n0) =
                        make_float4(h[k][0].x, h[k][0].y, h[k][1].x, h[k][1].y);
                    if (j == 0)
                        p.cpdt[at] = dtsum[k];
                }
        }
        // a few steps at a time: their decays and inputs first, which depend on
        // nothing before them, then the recurrence
#pragma unroll 1
        for (int tb = 0; tb < TT; tb += U) {
            float2 a[U][K][2], b[U][K][2];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const float4 both = *reinterpret_cast<const float4 *>(&sh.sd[buf][tb + i][cl]);
                const float2 dd[K] = {make_float2(both.x, both.y), make_float2(both.z, both.w)};
                const float4 bv = *reinterpret_cast<const float4 *>(&sh.sB[buf][tb + i][n0]);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float2 dt2 = make_float2(dd[k].x, dd[k].x), du2 = make_float2(dd[k].y, dd[k].y);
                    a[i][k][0] = decay2(dt2, A2[k][0]);
                    a[i][k][1] = decay2(dt2, A2[k][1]);
                    b[i][k][0] = mul2(du2, make_float2(bv.x, bv.y));
                    b[i][k][1] = mul2(du2, make_float2(bv.z, bv.w));
                    if (!kY)
                        dtsum[k] += dd[k].x;
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                float4 cv = make_float4(0.f, 0.f, 0.f, 0.f);
                if (kC)
                    cv = *reinterpret_cast<const float4 *>(&sh.sC[buf][tb + i][n0]);
                const float2 c0 = make_float2(cv.x, cv.y), c1 = make_float2(cv.z, cv.w);
                float part[K];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    h[k][0] = fma2(a[i][k][0], h[k][0], b[i][k][0]);
                    h[k][1] = fma2(a[i][k][1], h[k][1], b[i][k][1]);
                    if (kY) {
                        const float2 s = fma2(h[k][0], c0, mul2(h[k][1], c1));
                        part[k] = s.x + s.y;
                    }
                    if (kR) {
                        const float g = sh.sg[buf][tb + i][cl + k];
                        const float2 g2 = make_float2(g, g);
                        q[k][0] = mul2(q[k][0], a[i][k][0]);
                        q[k][1] = mul2(q[k][1], a[i][k][1]);
                        R[k][0] = fma2(q[k][0], mul2(g2, c0), R[k][0]);
                        R[k][1] = fma2(q[k][1], mul2(g2, c1), R[k][1]);
                    }
                }
                if (kY)
                    *reinterpret_cast<float2 *>(&sh.sy[buf][tb + i][j][cl]) = make_float2(part[0], part[1]);
            }
        }
        block_barrier(T::THREADS);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (cl + k >= w.nc)
            break;
        const int64_t hc = w.c0 + cl + k;
        const float4 out = make_float4(h[k][0].x, h[k][0].y, h[k][1].x, h[k][1].y);
        if (kY) {
            if (p.hT && w.chunk == p.chunks - 1)
                store_states(p.hT + (w.b * p.H + hc) * p.N, n0, p.N, p.vecState, out);
        } else {
            const int64_t at = (w.chunk * p.B + w.b) * p.H + hc;
            *reinterpret_cast<float4 *>(p.e + at * NP + n0) = out;
            if (j == 0)
                p.dts[at] = dtsum[k];
            if (kR)
                *reinterpret_cast<float4 *>(p.r + at * NP + n0) =
                    make_float4(R[k][0].x, R[k][0].y, R[k][1].x, R[k][1].y);
        }
    }
}

// Joins the chunks: e[c] becomes the state that enters chunk c (blockIdx.y = 0),
// r[c] the gradient that enters it from the right (blockIdx.y = 1). One thread
// per four states of a channel; a batch of chunks is loaded ahead of the
// recurrence over them.
__global__ void __launch_bounds__(128) mcc1d_ssm_scan_join(const ScanParams p, int NL)
{
    constexpr int K = 8;
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    const int64_t rows = p.B * p.H;
    if (i >= rows * NL)
        return;
    const int64_t row = i / NL;
    const int n0 = 4 * (int)(i - row * NL), NP = 4 * NL;
    const float4 A = load_states(p.A + row % p.H * p.N, n0, p.N, p.vecA);
    const float2 a0 = make_float2(A.x * kLog2e, A.y * kLog2e), a1 = make_float2(A.z * kLog2e, A.w * kLog2e);
    next_may_start();
    previous_done();
    const bool back = blockIdx.y == 1;
    float *const at = back ? p.r : p.e;
    const float *const first = back ? p.gfs : p.h0;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (first)
        s = load_states(first + row * p.N, n0, p.N, p.vecState);
    for (int64_t c0 = 0; c0 < p.chunks; c0 += K) {
        float4 v[K];
        float d[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c0 + k < p.chunks) {
                const int64_t c = (back ? p.chunks - 1 - c0 - k : c0 + k) * rows + row;
                v[k] = *reinterpret_cast<const float4 *>(at + c * NP + n0);
                d[k] = p.dts[c];
            }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (c0 + k < p.chunks) {
                const int64_t c = (back ? p.chunks - 1 - c0 - k : c0 + k) * rows + row;
                *reinterpret_cast<float4 *>(at + c * NP + n0) = s;
                const float2 lo = grown(make_float2(s.x, s.y), d[k], a0, make_float2(v[k].x, v[k].y));
                const float2 hi = grown(make_float2(s.z, s.w), d[k], a1, make_float2(v[k].z, v[k].w));
                s = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
    }
    if (back && p.gstate)
        store_states(p.gstate + row * p.N, n0, p.N, p.vecState, s);
}

constexpr int kStepThreads = 128;

// One token: a row of states in, moved on by one step, and out; the states'
// 8 N bytes per channel are what moves. Four states to a lane as above, so that
// neighbouring lanes move neighbouring 16 bytes. 256 rows of 4096 channels, N =
// 16: 27 us, 0.77 of the measured copy bandwidth (56 us with one row per
// thread, whose dt, gate and addresses all lanes of a channel worked out, 34
// with branches around the loads).
struct ScanStepParams {
    const uint16_t *u, *delta, *z, *Bm, *Cm;
    const float *A, *D, *dbias;
    float *state;
    const int32_t *slots;
    uint16_t *y;
    uint32_t ub, db, zb, Bb, Bg, Cb, Cg;   // strides below 2^31: products of 32 bits by 32
    int64_t rows;
    int32_t B, H, N, Hg, softplus;
};

template <int DT>
__device__ __forceinline__ float load16(const uint16_t *p)
{
    return unpack2<DT>((uint32_t)__ldg(p)).x;
}

// Four states of B or C, zeros past N.
template <int DT>
__device__ __forceinline__ void load_four(const uint16_t *row, int n0, int N, bool vec, float2 (&v)[2])
{
    uint32_t lo = 0u, hi = 0u;
    if (vec) {
        if (n0 < N) {
            const uint2 r = __ldg(reinterpret_cast<const uint2 *>(row + n0));
            lo = r.x;
            hi = r.y;
        }
    } else {
        lo = load_pair<false>(row + n0, n0 < N, n0 + 1 < N);
        hi = load_pair<false>(row + n0 + 2, n0 + 2 < N, n0 + 3 < N);
    }
    v[0] = unpack2<DT>(lo);
    v[1] = unpack2<DT>(hi);
}

// A thread takes R rows of one channel: A is read once, all rows' loads are in
// flight together, and what a row needs once per channel (dt, the gate, y) is
// done by one lane each instead of by all NL.
template <int NL>
constexpr int kStepRows = NL < 4 ? NL : 4;

// VEC: rows of the cache, A, B and C move four states at a time. Lanes past N
// and rows that are not there read where others do, write nothing and add
// nothing: loads without branches around them.
template <int DT, int NL, bool VEC>
__global__ void __launch_bounds__(kStepThreads) mcc1d_ssm_scan_step(const ScanStepParams p)
{
    constexpr int R = kStepRows<NL>;
    const int j = threadIdx.x % NL, lane = threadIdx.x & 31;
    const bool states = 4 * j < p.N;
    const int n0 = states ? 4 * j : 0;
    const int c = (int)(blockIdx.x * (kStepThreads / NL)) + (int)threadIdx.x / NL;
    const bool live = c < p.H;
    const int ch = live ? c : 0;
    const int b0 = (int)blockIdx.y * R, rows = p.B - b0 < R ? p.B - b0 : R;
    const uint32_t g = p.Hg == p.H ? 0 : ch / p.Hg, in_row = (uint32_t)(ch * p.N), row_size = (uint32_t)(p.H * p.N);
    const uint16_t *Bg = p.Bm + (uint64_t)g * p.Bg, *Cg = p.Cm + (uint64_t)g * p.Cg;

    float *at[R];
    bool on[R];
    float4 h[R];
    float2 B[R][2], C[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t b = b0 + (r < rows ? r : 0);
        const int32_t slot = p.slots ? p.slots[b] : (int32_t)b;
        on[r] = r < rows && slot >= 0 && slot < p.rows;
        at[r] = p.state + (uint64_t)(uint32_t)(on[r] ? slot : 0) * row_size + in_row;
        h[r] = load_states(at[r], n0, p.N, VEC);
        load_four<DT>(Bg + (uint64_t)b * p.Bb, n0, p.N, VEC, B[r]);
        load_four<DT>(Cg + (uint64_t)b * p.Cb, n0, p.N, VEC, C[r]);
    }
    const float4 A = load_states(p.A + in_row, n0, p.N, VEC);
    // this lane's own row
    const int own = j < R ? j : 0;
    const bool mine = live && j < R && own < rows;
    const uint32_t bm = b0 + (own < rows ? own : 0);
    float dt = load16<DT>(p.delta + (uint64_t)bm * p.db + ch) + (p.dbias ? p.dbias[ch] : 0.f);
    const float uv = load16<DT>(p.u + (uint64_t)bm * p.ub + ch);
    const float zv = p.z ? load16<DT>(p.z + (uint64_t)bm * p.zb + ch) : 0.f;
    const float D = p.D ? p.D[ch] : 0.f;
    if (p.softplus)
        dt = softplus(dt);
    const float dl = dt * kLog2e, du = dt * uv;

    float part[R];
    bool there = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float dlr = __shfl_sync(0xFFFFFFFFu, dl, r, NL), dur = __shfl_sync(0xFFFFFFFFu, du, r, NL);
        const float2 dl2 = make_float2(dlr, dlr), du2 = make_float2(dur, dur);
        const float2 o0 = fma2(decay2(dl2, make_float2(A.x, A.y)), make_float2(h[r].x, h[r].y), mul2(du2, B[r][0]));
        const float2 o1 = fma2(decay2(dl2, make_float2(A.z, A.w)), make_float2(h[r].z, h[r].w), mul2(du2, B[r][1]));
        if (on[r] && live && states)
            store_states(at[r], n0, p.N, VEC, make_float4(o0.x, o0.y, o1.x, o1.y));
        const float2 s = fma2(o0, C[r][0], mul2(o1, C[r][1]));
        part[r] = states ? s.x + s.y : 0.f;
        there = r == own ? on[r] : there;
    }
    lanes_sum<R, NL, 1, 1>(part, lane);
    float y = fmaf(D, uv, part[0]);
    if (p.z)
        y *= zv * sigmoid(zv);
    if (mine)
        p.y[(uint64_t)bm * p.H + ch] = there ? (uint16_t)pack2<DT>(make_float2(y, 0.f)) : (uint16_t)0;
}

bool aligned(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

template <class T, int DT, int MODE, bool PAIRS>
int32_t launch_tile(const ScanParams &p, cudaStream_t s)
{
    constexpr int bytes = (int)sizeof(ScanShared<T, MODE>);
    static SharedReady ready;
    if (!ready.set((const void *)mcc1d_ssm_scan<T, DT, MODE, PAIRS>, bytes))
        return kErrCuda;
    return launch_as(MODE == kOutputs && p.chunks > 1, mcc1d_ssm_scan<T, DT, MODE, PAIRS>, scan_launch_grid(p), T::THREADS, bytes, s, p);
}

template <class T, int MODE>
int32_t run_tile(const ScanParams &p, int dtype, cudaStream_t s)
{
    if (dtype == 0)
        return p.pairs ? launch_tile<T, 0, MODE, true>(p, s) : launch_tile<T, 0, MODE, false>(p, s);
    return p.pairs ? launch_tile<T, 1, MODE, true>(p, s) : launch_tile<T, 1, MODE, false>(p, s);
}

template <template <int> class Tile, int MODE>
int32_t run_scan(const ScanParams &p, int dtype, int nl, cudaStream_t s)
{
    switch (nl) {
    case 1: return run_tile<Tile<1>, MODE>(p, dtype, s);
    case 2: return run_tile<Tile<2>, MODE>(p, dtype, s);
    case 4: return run_tile<Tile<4>, MODE>(p, dtype, s);
    case 8: return run_tile<Tile<8>, MODE>(p, dtype, s);
    default: return run_tile<Tile<16>, MODE>(p, dtype, s);
    }
}

template <int DT, bool VEC>
int32_t run_step(const ScanStepParams &p, int nl, cudaStream_t s)
{
    const int per = kStepThreads / nl, rows = nl < 4 ? nl : 4;
    const dim3 grid((unsigned)((p.H + per - 1) / per), (unsigned)((p.B + rows - 1) / rows));
    switch (nl) {
    case 1: return launch(mcc1d_ssm_scan_step<DT, 1, VEC>, grid, kStepThreads, 0, s, p);
    case 2: return launch(mcc1d_ssm_scan_step<DT, 2, VEC>, grid, kStepThreads, 0, s, p);
    case 4: return launch(mcc1d_ssm_scan_step<DT, 4, VEC>, grid, kStepThreads, 0, s, p);
    case 8: return launch(mcc1d_ssm_scan_step<DT, 8, VEC>, grid, kStepThreads, 0, s, p);
    default: return launch(mcc1d_ssm_scan_step<DT, 16, VEC>, grid, kStepThreads, 0, s, p);
    }
}

uint64_t take(uint64_t &off, uint64_t bytes)
{
    const uint64_t at = off;
    off = (off + bytes + 255u) & ~(uint64_t)255u;
    return at;
}

ScanPlan shape_plan(const mcc1d_scan_args &a)
{
    ScanPlan p = {};
    p.nl = 1;
    while (4 * p.nl < a.N)
        p.nl *= 2;
    p.np = 4 * p.nl;
    return p;
}

ScanGrid scan_grid(int64_t H, int64_t G, int cb)
{
    ScanGrid g;
    g.blocks_per_group = (int32_t)((H / G + cb - 1) / cb);
    g.blocks = G * g.blocks_per_group;
    return g;
}

// Channels per block and rows per tile.
template <template <int> class Tile>
void tile_shape(int nl, int &cb, int &tt)
{
    switch (nl) {
    case 1: cb = Tile<1>::CB, tt = Tile<1>::TT; break;
    case 2: cb = Tile<2>::CB, tt = Tile<2>::TT; break;
    case 4: cb = Tile<4>::CB, tt = Tile<4>::TT; break;
    case 8: cb = Tile<8>::CB, tt = Tile<8>::TT; break;
    default: cb = Tile<16>::CB, tt = Tile<16>::TT; break;
    }
}

// Cuts the time axis into at most `most` chunks. The machine holds kSlots
// blocks at once (four per SM; the backward's first pass three), and a chunk
// costs about kChunkTiles tiles besides its own (setup, the join): the fewest
// waves of the fewest tiles, of more than `waves_above` waves where that can be
// had. The backward asks for more than two, since its passes hold different
// numbers of blocks and two waves of one are ragged in the other: 1024 x 8 x
// 2048 takes 503 us in 512 blocks a pass, 434 in 1024 and 429 in the 1792 that
// it gets. Where `most` chunks make no more than two waves they are taken
// without comparing costs: 509 x 2 x 768 takes 39 us in 32 chunks, 42 in 16 and
// 64 in 8. In between the rule can miss: 2048 x 2 x 1024 takes 127 us in the
// 43 chunks that it gets and 124 in 32.
void cut(ScanPlan &p, int64_t rows, int64_t most, int64_t waves_above)
{
    constexpr int64_t kSlots = 152 * 4, kChunkTiles = 2;
    most = std::min(std::max<int64_t>(most, 1), p.tiles);
    int64_t best = 0, chunks = 1;
    auto consider = [&](int64_t c) {
        if (c < 1 || c > most || (c < most && rows * c <= kSlots * waves_above))
            return;
        const int64_t cost = (rows * c + kSlots - 1) / kSlots * ((p.tiles + c - 1) / c + kChunkTiles);
        if (best == 0 || cost < best) {
            best = cost;
            chunks = c;
        }
    };
    for (int64_t c = 1; c <= 4; ++c)
        consider(c);
    for (int64_t waves = 1; waves <= 7; ++waves)
        consider(std::min(kSlots * waves / rows, most));
    p.tiles_per_chunk = (p.tiles + chunks - 1) / chunks;
    p.chunks = (p.tiles + p.tiles_per_chunk - 1) / p.tiles_per_chunk;
}

}  // namespace

ScanPlan scan_plan(const mcc1d_scan_args &a)
{
    ScanPlan p = shape_plan(a);
    // Cutting the time axis computes the states twice and costs two launches.
    // One pass against chunks, us: 256 blocks (2048 x 8 x 1024) 146 and 163, 192
    // (2048 x 6 x 1024) 140 and 125, 128 (2048 x 4 x 1024) 117 and 95; short
    // sequences: 8 tiles (128 x 4 x 1024) 12.4 and 14.5, 16 tiles (256 x 2 x 1024)
    // 18.8 and 14.6.
    int cb;
    tile_shape<OutTile>(p.nl, cb, p.tt);
    p.tiles = (a.S + p.tt - 1) / p.tt;
    p.grid = scan_grid(a.H, a.G, cb);
    const int64_t rows = p.grid.blocks * a.B;
    cut(p, rows, rows >= 220 || p.tiles < 12 ? 1 : p.tiles / 2, 0);
    p.most_blocks = rows * p.chunks;
    uint64_t off = 0;
    const uint64_t ch = (uint64_t)(a.B * a.H);
    if (p.chunks > 1) {
        p.off_e = take(off, (uint64_t)p.chunks * ch * p.np * 4);
        p.off_dt = take(off, (uint64_t)p.chunks * ch * 4);
    }
    p.bytes = off;
    return p;
}

ScanPlan scan_bwd_plan(const mcc1d_scan_bwd_args &ba)
{
    const mcc1d_scan_args &a = ba.fwd;
    ScanPlan p = shape_plan(a);
    int cb;
    tile_shape<BwdTile>(p.nl, cb, p.tt);
    p.tiles = (a.S + p.tt - 1) / p.tt;
    p.grid = scan_grid(a.H, a.G, cb);
    const int64_t rows = p.grid.blocks * a.B;
    cut(p, rows, p.tiles, 2);
    p.most_blocks = rows * p.chunks;
    uint64_t off = 0;
    const uint64_t ch = (uint64_t)(a.B * a.H);
    p.off_e = take(off, (uint64_t)p.chunks * ch * p.np * 4);
    p.off_r = take(off, (uint64_t)p.chunks * ch * p.np * 4);
    p.off_dt = take(off, (uint64_t)p.chunks * ch * 4);
    p.off_cp = take(off, (uint64_t)p.tiles * ch * p.np * 4);
    p.off_cpdt = take(off, (uint64_t)p.tiles * ch * 4);
    p.off_ga = take(off, (uint64_t)p.chunks * ch * p.np * 4);
    p.off_gd = take(off, (uint64_t)p.chunks * ch * 8);
    p.off_bc = take(off, (uint64_t)(a.S * a.B) * (uint64_t)p.grid.blocks * 2u * p.np * 4);
    p.bytes = off;
    return p;
}

static ScanParams scan_params(const mcc1d_scan_args &a, const ScanPlan &pl, uint8_t *ws)
{
    ScanParams p = {};
    p.u = (const uint16_t *)a.u;
    p.delta = (const uint16_t *)a.delta;
    p.z = (const uint16_t *)a.z;
    p.Bm = (const uint16_t *)a.B_;
    p.Cm = (const uint16_t *)a.C;
    p.A = a.A;
    p.D = a.D;
    p.dbias = a.delta_bias;
    p.h0 = a.state;
    p.lengths = a.lengths;
    p.y = (uint16_t *)a.y;
    p.hT = a.final_state;
    p.us = a.u_strides[0], p.ub = a.u_strides[1];
    p.ds = a.delta_strides[0], p.db = a.delta_strides[1];
    p.zs = a.z ? a.z_strides[0] : 0, p.zb = a.z ? a.z_strides[1] : 0;
    p.Bs = a.B_strides[0], p.Bb = a.B_strides[1], p.Bg = a.B_strides[2];
    p.Cs = a.C_strides[0], p.Cb = a.C_strides[1], p.Cg = a.C_strides[2];
    p.S = a.S;
    p.B = a.B;
    p.H = a.H;
    p.N = (int32_t)a.N;
    p.G = (int32_t)a.G;
    p.Hg = (int32_t)(a.H / a.G);
    p.grid = pl.grid;
    p.tiles = pl.tiles;
    p.tiles_per_chunk = pl.tiles_per_chunk;
    p.chunks = pl.chunks;
    p.softplus = (a.flags & MCC1D_SOFTPLUS) != 0;
    const uintptr_t any = (uintptr_t)a.u | (uintptr_t)a.delta | (uintptr_t)a.z | (uintptr_t)a.y;
    const int64_t steps = p.us | p.ub | p.ds | p.db | p.zs | p.zb | a.H | p.Hg;
    p.pairs = (any & 3u) == 0 && (steps & 1) == 0;
    const uintptr_t bca = (uintptr_t)a.B_ | (uintptr_t)a.C;
    const int64_t bcs = p.Bs | p.Bb | p.Bg | p.Cs | p.Cb | p.Cg | a.N;
    p.bcpairs = (bca & 3u) == 0 && (bcs & 1) == 0;
    p.bc8 = (bca & 15u) == 0 && (bcs & 7) == 0;
    p.vecA = a.N % 4 == 0 && aligned(a.A, 16);
    p.vecState = a.N % 4 == 0 && aligned(a.state, 16) && aligned(a.final_state, 16);
    p.e = (float *)(ws + pl.off_e);
    p.r = (float *)(ws + pl.off_r);
    p.dts = (float *)(ws + pl.off_dt);
    p.cp = (float *)(ws + pl.off_cp);
    p.cpdt = (float *)(ws + pl.off_cpdt);
    p.ga = (float *)(ws + pl.off_ga);
    p.gd = (float *)(ws + pl.off_gd);
    p.bc = (float *)(ws + pl.off_bc);
    return p;
}

static int32_t join(const ScanParams &p, int nl, bool grad, cudaStream_t s)
{
    const dim3 grid((unsigned)((p.B * p.H * nl + 127) / 128), grad ? 2 : 1);
    return launch_as(true, mcc1d_ssm_scan_join, grid, 128, 0, s, p, nl);
}

int32_t launch_scan(const mcc1d_scan_args &a, const ScanPlan &pl, void *workspace, cudaStream_t stream)
{
    const ScanParams p = scan_params(a, pl, (uint8_t *)workspace);
    if (p.chunks > 1) {
        int32_t st = run_scan<OutTile, kSummary>(p, a.dtype, pl.nl, stream);
        if (st == kOk)
            st = join(p, pl.nl, false, stream);
        if (st != kOk)
            return st;
    }
    return run_scan<OutTile, kOutputs>(p, a.dtype, pl.nl, stream);
}

int32_t launch_scan_bwd(const mcc1d_scan_bwd_args &a, const ScanPlan &pl, void *workspace, cudaStream_t stream)
{
    ScanParams p = scan_params(a.fwd, pl, (uint8_t *)workspace);
    p.gy = (const uint16_t *)a.grad_y;
    p.gs = a.grad_y_strides[0];
    p.gb = a.grad_y_strides[1];
    p.gfs = a.grad_final_state;
    p.gu = (uint16_t *)a.grad_u;
    p.gdelta = (uint16_t *)a.grad_delta;
    p.gz = (uint16_t *)a.grad_z;
    p.gstate = a.grad_state;
    const uintptr_t any = (uintptr_t)a.grad_y | (uintptr_t)a.grad_u | (uintptr_t)a.grad_delta | (uintptr_t)a.grad_z |
                          (uintptr_t)a.fwd.u | (uintptr_t)a.fwd.delta | (uintptr_t)a.fwd.z;
    const int64_t steps = p.us | p.ub | p.ds | p.db | p.zs | p.zb | p.gs | p.gb | p.H | p.Hg;
    p.pairs = (any & 3u) == 0 && (steps & 1) == 0;
    p.vecState = a.fwd.N % 4 == 0 && aligned(a.fwd.state, 16) && aligned(a.grad_final_state, 16) &&
                 aligned(a.grad_state, 16);
    int32_t st = run_scan<BwdTile, kSummaryGrad>(p, a.fwd.dtype, pl.nl, stream);
    if (st == kOk)
        st = join(p, pl.nl, true, stream);
    if (st != kOk)
        return st;
    return launch_scan_bwd_main(p, pl, a, stream);
}

int32_t launch_scan_step(const mcc1d_scan_step_args &a, cudaStream_t stream)
{
    ScanStepParams p;
    p.u = (const uint16_t *)a.u;
    p.delta = (const uint16_t *)a.delta;
    p.z = (const uint16_t *)a.z;
    p.Bm = (const uint16_t *)a.B_;
    p.Cm = (const uint16_t *)a.C;
    p.A = a.A;
    p.D = a.D;
    p.dbias = a.delta_bias;
    p.state = a.state;
    p.slots = a.slots;
    p.y = (uint16_t *)a.y;
    p.ub = (uint32_t)a.u_stride;
    p.db = (uint32_t)a.delta_stride;
    p.zb = (uint32_t)a.z_stride;
    p.Bb = (uint32_t)a.B_strides[0], p.Bg = (uint32_t)a.B_strides[1];
    p.Cb = (uint32_t)a.C_strides[0], p.Cg = (uint32_t)a.C_strides[1];
    p.rows = a.cache_rows;
    p.B = (int32_t)a.B;
    p.H = (int32_t)a.H;
    p.N = (int32_t)a.N;
    p.Hg = (int32_t)(a.H / a.G);
    p.softplus = (a.flags & MCC1D_SOFTPLUS) != 0;
    const bool vec = a.N % 4 == 0 && aligned(a.A, 16) && aligned(a.state, 16) && aligned(a.B_, 8) && aligned(a.C, 8) &&
                     ((p.Bb | p.Bg | p.Cb | p.Cg) & 3) == 0;
    int nl = 1;
    while (4 * nl < a.N)
        nl *= 2;
    if (a.dtype == 0)
        return vec ? run_step<0, true>(p, nl, stream) : run_step<0, false>(p, nl, stream);
    return vec ? run_step<1, true>(p, nl, stream) : run_step<1, false>(p, nl, stream);
}

}  // namespace mcc1d
