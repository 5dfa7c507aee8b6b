// delta_chunks.cu - the gated delta rule over prompts, a chunk of 64 tokens at
// a time, on the tensor cores.
//
// A block has one head's state [V,K], up to 128 rows of it, a row to four
// threads that share its columns: everything that goes along a row (decays,
// sums, scales, rounding to two fp16 terms) stays in them, and the state itself
// in their registers, in fp32. With the factors of delta_prepare.cu, a chunk is
//   X = S K^T        R = b V - e^c X          (A: the state, from tensor memory)
//   U = R T^T        Y = e^c S Q^T + R (PT)^T
//   S = e^c(end) S + (U e^(c(end)-c)) K
// with tokens along the columns; R is taken without each token's growth, which T's
// and P T's columns put back (growth_of in delta_prepare.cu). Operands in tensor
// memory are two fp16 terms of fp32 rows scaled by a power of two, 22 bits; K and Q
// are exact in fp16 (rows scaled by a power of two), so those products take two
// terms and those with T and P T three. Sums are fp32.
//
// The chunks of one head follow on one another, X - R - U - S, and bound the
// kernel: the products' time and the conversions between them, for which a
// scheduler has four warps of rows: 4096 tokens of 8 x 16 heads of 128 x 128 take
// 243 us, 3.8 us a chunk; q, k, v, y and the factors would take 1.9 at the
// copy bandwidth. Y is taken in the gaps and leaves through
// warps of its own. Warps 0 to 15 hold the rows, 16 to 19 write Y, 20 issues the
// products, 21 copies the tokens of the chunk after the next, 22 to 27 make
// panels of the next one's and look for values that are not finite (looked for by the
// rows' threads, on the chain, it cost 8 us of 34 over eight chunks).
#include <limits.h>

#include <utility>

#include "delta_chunks.cuh"

namespace mcc1d {

namespace {

constexpr int kTiles = 3, kPrepareds = 2;      // chunks whose tokens, and whose prepared panels, are there or on their way
// Registers by warpgroup: rows (four), Y, and two for the rest.
constexpr int kRegRows = 80, kRegY = 64, kRegRest = 56, kRegLaunch = 72;
static_assert(kParts * kRegRows + kRegY + 2 * kRegRest <= kThreads / 128 * kRegLaunch, "what the block is launched with");

struct ChunkParams {
    CUtensorMap map_q, map_k, map_v;    // where rows can be copied as tiles
    DeltaParams d;
    const uint8_t *prepared;
    int32_t record;           // bytes of a chunk's there
    int64_t chunks;
    int32_t tiles;            // of 128 rows of V
    bool vectors_q, vectors_k, vectors_v, vectors_s;
    bool pairs_y;             // two rows of y are one word
    Segments seg;
};

// Tokens: 64 keys of K's rows, then of Q's, then the next 64 keys; V as it is, 64
// values of its rows, then the next 64.
template <int KP>
struct Tile {
    static constexpr int kPanels = KP / 64 * kPanelBytes;
    static constexpr int K = 0, Q = kPanelBytes, V = 2 * kPanels, kBytes = V + kRows / 64 * kPanelBytes;
    static constexpr int kAll = kTiles * kBytes;
};
constexpr int kPreparedBytes = kForwardBytes;

// Columns of tensor memory: sums, then operands (pairs of fp16). The state's
// update is summed over X and U.
enum { kUpdate = 0, kX = 0, kU = 64, kQS = 128, kPR = 192, kSHi = 256, kSLo = 320, kWHi = 384, kWLo = 416, kVHi = 448, kVLo = 480, kColumns = 512 };

struct ChunkShared {
    uint64_t tiles[kTiles], full[kTiles], tile_free[kTiles], prepared[kPrepareds], prepared_free[kPrepareds], x, r, u, v, y, s, end, out;
    float of_s[2][kRows], of_r[2][kRows];       // of the last two chunks: what rows' terms are multiplied by
    float of_y[4][2 * kC];                      // the factors of Y of the last four chunks
    float most[kParts][kRows], most_v[kParts][kRows], sum_u[kParts][kRows];      // of the parts of a row
    int bad[kRows];                              // the first token whose value is not finite, of rows that have one
    uint32_t tmem, failed;
};

// A chunk's rows of q or k made scaled fp16 where they lie in their panels (or
// come from global memory). A thread has one piece of every STEPth row.
template <int DT, int KP>
__device__ __forceinline__ void make_panels(uint8_t *panels, const uint16_t *from, int64_t step, const float *scales, int K, bool vectors, int n, int thread)
{
    constexpr int PIECES = KP / 8, STEP = kLoadThreads / PIECES;
    static_assert(kLoadThreads % PIECES == 0, "whole rows");
    const int piece = thread % PIECES, live = K - 8 * piece;
    panels += (piece / 8) * 2 * kPanelBytes;
#pragma unroll 2
    for (int t = thread / PIECES; t < kC; t += STEP) {
        uint8_t *at = panels + panel_at(t, piece % 8);
        const uint4 v = piece_of(at, from + t * step + 8 * piece, vectors, t < n ? live : 0);
        const float2 f = make_float2(scales[t], scales[t]);
        *reinterpret_cast<uint4 *>(at) = make_uint4(pack_half2(mul2(unpack2<DT>(v.x), f)), pack_half2(mul2(unpack2<DT>(v.y), f)),
                                                    pack_half2(mul2(unpack2<DT>(v.z), f)), pack_half2(mul2(unpack2<DT>(v.w), f)));
    }
}

// A chunk's rows of v where they were not copied, and zeros behind their end.
__device__ __forceinline__ void fill_values(uint8_t *values, const uint16_t *from, int64_t step, int V, bool vectors, int n, int thread)
{
    constexpr int PIECES = kRows / 8;
    const int piece = thread % PIECES, live = V - 8 * piece;
#pragma unroll 1
    for (int t = thread / PIECES + (vectors && live > 0 ? n / (kLoadThreads / PIECES) * (kLoadThreads / PIECES) : 0); t < kC; t += kLoadThreads / PIECES)
        if (!vectors || t >= n || live <= 0)
            *reinterpret_cast<uint4 *>(values + (piece / 8) * kPanelBytes + t * 128 + 16 * (piece % 8)) =
                piece_of(nullptr, from + t * step + 8 * piece, false, t < n && !vectors ? live : 0);
}

// Values that are not finite become zeros where they lie: in a row's operands they
// would, times zeros of T, make NaN of earlier tokens too. A row's first of them is
// noted (`first`: the chunk's first token), and its outputs from there on and its state
// become NaN. The threads have the pieces that they have in fill_values.
template <int DT>
__device__ __forceinline__ void leave_out(uint8_t *values, int V, int n, int first, int *bad, int thread)
{
    constexpr int PIECES = kRows / 8, STEP = kLoadThreads / PIECES;
    constexpr uint32_t INF = DT == 0 ? 0x7F80u : 0x7C00u;
    const int piece = thread % PIECES;
    if (V - 8 * piece <= 0)
        return;
    uint8_t *at = values + (piece / 8) * kPanelBytes + 16 * (piece % 8);
    uint32_t most = 0u;           // magnitudes are in the order of their bits
#pragma unroll 2
    for (int t = thread / PIECES; t < n; t += STEP) {
        const uint4 v = *reinterpret_cast<const uint4 *>(at + t * 128);
        most = __vmaxu2(__vmaxu2(most, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
    }
    if ((most & 0xFFFFu) < INF && most >> 16 < INF)
        return;
#pragma unroll 1
    for (int t = thread / PIECES; t < n; t += STEP)
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
            uint16_t &x = reinterpret_cast<uint16_t *>(at + t * 128)[e];
            if ((x & 0x7FFFu) >= INF)
                x = 0, atomicMin(bad + 8 * piece + e, first + t);
        }
}

// ------------------------------------------------------------------ the rows
template <int DT, int KP>
__device__ __forceinline__ void hold_rows(const ChunkParams &cp, ChunkShared &sh, const uint8_t *tiles, const Part &pt, int64_t n)
{
    typedef Tile<KP> Tl;
    constexpr int HK = KP / kParts, HC = kC / kParts, UNIT = HK < 32 ? HK : 32;
    const DeltaParams &p = cp.d;
    const int warp = threadIdx.x / 32, r = threadIdx.x % kRows, part = warp / 4, row = pt.v0 + r;
    const int64_t BH = (int64_t)p.B * p.H, chunks = pt.chunks, item = pt.item;
    const bool mine = row < pt.rows;
    const uint32_t lanes = sh.tmem + ((uint32_t)(32 * (warp % 4)) << 16);
    float s[HK];             // the state times `scale_s`, a power of two
    {
        const float *from = pt.from + (int64_t)row * p.K + part * HK;
#pragma unroll
        for (int k = 0; k < HK; ++k)
            s[k] = pt.from && mine && part * HK + k < p.K ? from[k] : pt.unit && row == part * HK + k ? 1.f : 0.f;
    }
    float scale_s;
    // Scales come from bounds, so that no thread waits for its row's other parts
    // where the products wait for it: terms keep 22 bits of a row up to 2^17 below
    // its bound. The state's largest value is known a phase late, the sum of a
    // row's |U| in time.
    sh.most[part][r] = most_of(s);
    rows_meet();
    scale_s = scale_for(most_of_parts(sh.most, r));
    rows_meet();
#pragma unroll
    for (int k = 0; k < HK; ++k)
        s[k] *= scale_s;
    const uint32_t terms_s = lanes + kSHi + HK / 2 * part, terms_w = lanes + kWHi + HC / 2 * part, terms_v = lanes + kVHi + HC / 2 * part;
    if (chunks > 0) {
        sh.of_s[0][r] = inverse_scale(scale_s);
#pragma unroll
        for (int c = 0; c < HK; c += UNIT)
            put_terms<UNIT>(s + c, terms_s + c / 2, terms_s + (kSLo - kSHi) + c / 2);
        terms_done(sh.s);
    }
    bool ok = true;          // no wait gave up
    for (int64_t i = 0;; ++i) {
        const uint32_t parity = (uint32_t)(i & 1);
        if (!ok)
#pragma unroll
            for (int k = 0; k < HK; ++k)
                s[k] = __uint_as_float(0x7FFFFFFFu);
        if (i < chunks && p.kept.states && mine) {
            const float of = inverse_scale(scale_s);
            float *to = p.kept.states + (((pt.first + i) * BH + item) * p.K + part * HK) * p.kept.Vp + row;
#pragma unroll
            for (int k = 0; k < HK; ++k, to += p.kept.Vp)
                if (part * HK + k < p.K)
                    *to = s[k] * of;
        }
        if (i >= chunks && pt.to && mine)
            write_row<HK>(pt.to + (int64_t)row * p.K, part * HK, p.K, cp.vectors_s, s, inverse_scale(scale_s));
        if (i >= chunks)
            break;
        const uint8_t *prepared = tiles + Tl::kAll + (i % kPrepareds) * kPreparedBytes;
        const float *f = reinterpret_cast<const float *>(prepared + kAtFactors), *ends = f + kFactorEnd * kC;
        const uint16_t *v = reinterpret_cast<const uint16_t *>(tiles + (i % kTiles) * Tl::kBytes + Tl::V + (r / 64) * kPanelBytes) + part * HC * 64 + r % 64;
        f += part * HC;
        // the products wait for the chunk's tiles too, but this thread reads some itself
        ok = warp_wait(sh.full[i % kTiles], (uint32_t)(i / kTiles) & 1);
        float most_v = 0.f;          // as R has them
        uint32_t pairs[HC / 2];      // of tokens
#pragma unroll
        for (int t = 0; t < HC; t += 2) {
            pairs[t / 2] = v[t * 64] | (uint32_t)v[(t + 1) * 64] << 16;
            const float2 x = mul2(*reinterpret_cast<const float2 *>(f + kFactorB * kC + t), unpack2<DT>(pairs[t / 2]));
            most_v = fmaxf(most_v, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
        sh.most[part][r] = most_of(s);
        sh.most_v[part][r] = most_v;
        rows_meet();
        if (sh.failed) {         // all rows leave together; theirs are NaN
            ok = false;
            i = chunks - 1;
            continue;
        }
        const float of_s = inverse_scale(scale_s), most_s = most_of_parts(sh.most, r) * of_s;
        const float bound_r = fmaf(ends[kEndOfState], most_s, most_of_parts(sh.most_v, r));
        // times b 2^17 at most, and still a number; rows below 2^-86 are held to 2^-126 so
        const float scale_r = fminf(scale_for(bound_r), 0x1p100f), of_r = inverse_scale(scale_r);
        const float scale_u = scale_for(bound_r * ends[kEndOfR]), of_u = inverse_scale(scale_u), end = ends[kEndDecay];
        if (part == 0)
            sh.of_r[parity][r] = of_r;
        ok = ok && warp_wait(sh.x, parity);
        tmem_fence_after();
        const float2 mx = make_float2(-of_s * scale_r, -of_s * scale_r), mv = make_float2(scale_r, scale_r);
#pragma unroll
        for (int t0 = 0; t0 < HC; t0 += 16) {
            uint32_t raw[16];
            float x[16];
            tmem_load(lanes + kX + HC * part + t0, raw);
            tmem_wait(raw);
#pragma unroll
            for (int t = 0; t < 16; t += 2) {
                const float2 bt = *reinterpret_cast<const float2 *>(f + kFactorB * kC + t0 + t), ft = *reinterpret_cast<const float2 *>(f + kFactorX * kC + t0 + t);
                const float2 a = fma2(mul2(ft, mx), make_float2(__uint_as_float(raw[t]), __uint_as_float(raw[t + 1])),
                                      mul2(mul2(bt, mv), unpack2<DT>(pairs[(t0 + t) / 2])));
                x[t] = a.x, x[t + 1] = a.y;
            }
            put_terms<16>(x, terms_w + t0 / 2, terms_w + (kWLo - kWHi) + t0 / 2);
        }
        terms_done(sh.r);
        ok = ok && warp_wait(sh.u, parity);
        tmem_fence_after();
        float2 sum_u = make_float2(0.f, 0.f);
        const float2 mu = make_float2(of_r * scale_u, of_r * scale_u);
#pragma unroll
        for (int t0 = 0; t0 < HC; t0 += 16) {
            uint32_t raw[16];
            float x[16];
            tmem_load(lanes + kU + HC * part + t0, raw);
            tmem_wait(raw);
            if (p.kept.u && mine) {
                const int64_t at = (pt.first + i) * kC + part * HC + t0, step = BH * p.kept.Vp;
                float *to_u = p.kept.u + (at * BH + item) * p.kept.Vp + row;
#pragma unroll
                for (int t = 0; t < 16; ++t, to_u += step)
                    if (at + t < n)
                        *to_u = __uint_as_float(raw[t]) * (of_r * f[kFactorT * kC + t0 + t]);
            }
#pragma unroll
            for (int t = 0; t < 16; t += 2) {
                const float2 ft = *reinterpret_cast<const float2 *>(f + kFactorU * kC + t0 + t);
                const float2 a = mul2(mul2(ft, mu), make_float2(__uint_as_float(raw[t]), __uint_as_float(raw[t + 1])));
                sum_u = add2(sum_u, make_float2(fabsf(a.x), fabsf(a.y)));
                x[t] = a.x, x[t + 1] = a.y;
            }
            put_terms<16>(x, terms_v + t0 / 2, terms_v + (kVLo - kVHi) + t0 / 2);
        }
        sh.sum_u[part][r] = sum_u.x + sum_u.y;
        terms_done(sh.v);
        warp_arrive(sh.tile_free[i % kTiles]);
        warp_arrive(sh.prepared_free[i % kPrepareds]);
        rows_meet();     // for sum_u, while the products run
        // |S| <= e^c(end) |S| + sum of |U k|, and no |k| is above 2^16 as an operand
        const float before = scale_s;
        scale_s = scale_for(fmaf(fabsf(end), most_s, ((sh.sum_u[0][r] + sh.sum_u[1][r]) + (sh.sum_u[2][r] + sh.sum_u[3][r])) * of_u * 65536.f));
        const float kept = sh.bad[r] < (int)(pt.first + i + 1) * kC ? __uint_as_float(0x7FFFFFFFu) : end * inverse_scale(before) * scale_s;
        const float2 keep = make_float2(kept, kept), add = make_float2(of_u * scale_s, of_u * scale_s);
        if (part == 0)
            sh.of_s[parity ^ 1][r] = inverse_scale(scale_s);
        ok = ok && warp_wait(sh.end, parity);
        tmem_fence_after();
        if (!ok)
            sh.failed = 1;
#pragma unroll
        for (int c = 0; c < HK; c += UNIT) {
            uint32_t raw[UNIT];
            tmem_load(lanes + kUpdate + HK * part + c, raw);
            tmem_wait(raw);
#pragma unroll
            for (int k = 0; k < UNIT; k += 2) {
                const float2 o = fma2(add, make_float2(__uint_as_float(raw[k]), __uint_as_float(raw[k + 1])), mul2(keep, make_float2(s[c + k], s[c + k + 1])));
                s[c + k] = o.x, s[c + k + 1] = o.y;
            }
            if (i + 1 < chunks)
                put_terms<UNIT>(s + c, terms_s + c / 2, terms_s + (kSLo - kSHi) + c / 2);
        }
        if (i + 1 < chunks)
            terms_done(sh.s);
    }
}

// ------------------------------------------------------------------ Y
template <int DT>
__device__ __forceinline__ void write_y(const ChunkParams &cp, ChunkShared &sh, const Part &pt, int64_t n)
{
    const DeltaParams &p = cp.d;
    const int r = threadIdx.x % kRows, row = pt.v0 + r;
    const int64_t step = (int64_t)p.B * p.H * p.V, chunks = pt.chunks;
    const bool mine = row < p.V;
    const uint32_t lanes = sh.tmem + ((uint32_t)(32 * (threadIdx.x / 32 % 4)) << 16);
    uint16_t *to = p.y + pt.first * kC * step + (int64_t)pt.item * p.V + row;
    const bool odd = r & 1;
    uint16_t *pair = odd ? to + step - 1 : to;         // whole chunks come first
    int64_t i = 0;
    for (; i < chunks; ++i) {
        if (!warp_wait(sh.y, (uint32_t)(i & 1)))
            break;
        const float *fq = sh.of_y[i & 3], *fp = fq + kC;
        tmem_fence_after();
        const float2 of_s = make_float2(sh.of_s[i & 1][r], sh.of_s[i & 1][r]), of_r = make_float2(sh.of_r[i & 1][r], sh.of_r[i & 1][r]);
        const int64_t t1 = (pt.first + i) * kC;
        const int live = (int)(n - t1 < kC ? n - t1 : kC), rows = (int)(p.S - t1 < kC ? p.S - t1 : kC);
        const bool whole = cp.pairs_y && rows == kC && live == kC;
        const int good = sh.bad[r] - (int)t1;
#pragma unroll 1
        for (int t0 = 0; t0 < kC; t0 += 16) {
            uint32_t a[16], c[16], y[8];
            tmem_load(lanes + kQS + t0, a);
            tmem_load(lanes + kPR + t0, c);
            tmem_wait(a), tmem_wait(c);
            if (t0 == kC - 16) {
                tmem_fence_before();
                warp_arrive(sh.out);
            }
#pragma unroll
            for (int t = 0; t < 16; t += 2) {
                const float2 q = *reinterpret_cast<const float2 *>(fq + t0 + t), pr = *reinterpret_cast<const float2 *>(fp + t0 + t);
                y[t / 2] = pack2<DT>(fma2(mul2(pr, of_r), make_float2(__uint_as_float(c[t]), __uint_as_float(c[t + 1])),
                                          mul2(mul2(q, of_s), make_float2(__uint_as_float(a[t]), __uint_as_float(a[t + 1])))));
            }
            if (good < t0 + 16)
#pragma unroll
                for (int t = 0; t < 16; ++t)
                    if (t0 + t >= good)
                        y[t / 2] |= t % 2 ? 0x7FFF0000u : 0x00007FFFu;
            if (whole) {        // two rows of one token: even lanes the first, odd lanes the second
#pragma unroll
                for (int t = 0; t < 8; ++t, pair += 2 * step) {
                    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, y[t], 1);
                    if (mine)
                        *reinterpret_cast<uint32_t *>(pair) = odd ? __byte_perm(other, y[t], 0x7632) : __byte_perm(y[t], other, 0x5410);
                }
            } else {
                uint16_t *at = to + t0 * step;
#pragma unroll
                for (int t = 0; t < 16; ++t, at += step)
                    if (mine && t0 + t < rows)
                        *at = t0 + t < live ? (uint16_t)(y[t / 2] >> (16 * (t % 2))) : (uint16_t)0;
            }
        }
        to += kC * step;
    }
    if (mine)          // tokens behind the sequence; NaN where a wait gave up
        for (int64_t t = (pt.first + i) * kC, end = pt.last ? p.S : (pt.first + chunks) * kC; t < end; ++t, to += step)
            *to = i < chunks ? 0x7FFF : 0;
}

// ------------------------------------------------------------------ products
// One thread's, second terms first. Each of them is added with its last bits cut
// off, towards zero, so the fewer to a sum of full size the better: with first and
// second terms in turn states were 2e-7 too small (and the kernel took 225 us). `y`: those of Y too.
template <int KP>
__device__ __forceinline__ void issue_products(ChunkShared &sh, uint32_t tiles, int64_t chunks, bool y)
{
    typedef Tile<KP> Tl;
    constexpr uint32_t by_rows = mma_kind(kC, false), by_columns = mma_kind(KP, true);
    const uint32_t tmem = sh.tmem;
    const auto wait = [](uint64_t &bar, uint32_t parity) { return mbar_wait_bounded_inline(smem_u32(&bar), parity); };
    const auto with_state = [&](uint32_t d, uint32_t panels) {
#pragma unroll
        for (int j = 0; j < KP / 16; ++j)
            mma_ts(tmem + d, tmem + kSLo + 8 * j, desc_rows(panels + (j / 4) * 2 * kPanelBytes) + 2 * (j % 4), by_rows, j > 0);
#pragma unroll
        for (int j = 0; j < KP / 16; ++j)
            mma_ts(tmem + d, tmem + kSHi + 8 * j, desc_rows(panels + (j / 4) * 2 * kPanelBytes) + 2 * (j % 4), by_rows, true);
    };
    const auto with_r = [&](uint32_t d, uint32_t panels) {        // first terms, second ones behind them
#pragma unroll
        for (int j = 0; j < kC / 16; ++j) {
            mma_ts(tmem + d, tmem + kWHi + 8 * j, desc_rows(panels + kPanelBytes) + 2 * j, by_rows, j > 0);
            mma_ts(tmem + d, tmem + kWLo + 8 * j, desc_rows(panels) + 2 * j, by_rows, true);
        }
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ts(tmem + d, tmem + kWHi + 8 * j, desc_rows(panels) + 2 * j, by_rows, true);
    };
    for (int64_t i = 0; i < chunks; ++i) {
        const uint32_t parity = (uint32_t)(i & 1), tile = tiles + (uint32_t)(i % kTiles) * Tl::kBytes;
        const uint32_t prepared = tiles + Tl::kAll + (uint32_t)(i % kPrepareds) * kPreparedBytes;
        if (!wait(sh.full[i % kTiles], (uint32_t)(i / kTiles) & 1) || !wait(sh.s, parity))
            break;
        tmem_fence_after();
        with_state(kX, tile + Tl::K);
        mma_commit(smem_u32(&sh.x));
        if (y) {                   // while X becomes R, and U an operand
            if (!wait(sh.out, parity ^ 1))         // the Y before this one has been read
                break;
            tmem_fence_after();
            with_state(kQS, tile + Tl::Q);
        }
        if (!wait(sh.r, parity))
            break;
        tmem_fence_after();
        with_r(kU, prepared + kAtT);
        mma_commit(smem_u32(&sh.u));
        if (y) {
            with_r(kPR, prepared + kAtPT);
            mma_commit(smem_u32(&sh.y));
        }
        if (!wait(sh.v, parity))
            break;
        tmem_fence_after();
        const uint64_t k = desc_columns(tile + Tl::K, 2 * kPanelBytes);
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ts(tmem + kUpdate, tmem + kVLo + 8 * j, k + (uint64_t)(2048 * j >> 4), by_columns, j > 0);
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ts(tmem + kUpdate, tmem + kVHi + 8 * j, k + (uint64_t)(2048 * j >> 4), by_columns, true);
        mma_commit(smem_u32(&sh.end));
        mma_commit(smem_u32(&sh.tile_free[i % kTiles]));
        mma_commit(smem_u32(&sh.prepared_free[i % kPrepareds]));
    }
}

// ------------------------------------------------------------------ tiles
// One warp: a chunk's rows as tiles of 64 tokens and 64 values, up to three chunks
// ahead, and its prepared panels and factors.
template <int KP>
__device__ __forceinline__ void copy_tiles(const ChunkParams &cp, ChunkShared &sh, uint8_t *tiles, const Part &pt)
{
    typedef Tile<KP> Tl;
    const DeltaParams &p = cp.d;
    const int b = pt.item / p.H, h = pt.item % p.H, g = h / (p.H / p.G), v0 = pt.v0;
    const int64_t chunks = pt.chunks;
    const bool k = cp.vectors_k, q = cp.vectors_q && p.y, v = cp.vectors_v && !pt.unit;
    int64_t next = 0;          // whose tokens are to be asked for
    for (int64_t i = 0; i < chunks; ++i) {
        for (; next < chunks && next < i + kTiles; ++next) {
            if (next > i && !__all_sync(0xFFFFFFFFu, mbar_test(smem_u32(&sh.tile_free[next % kTiles]), (uint32_t)(next / kTiles + 1) & 1)))
                break;         // not free yet, and not what is waited for
            if (!warp_wait(sh.tile_free[next % kTiles], (uint32_t)(next / kTiles + 1) & 1))
                return;
            if (threadIdx.x % 32 == 0) {
                const uint32_t tile = smem_u32(tiles) + (uint32_t)(next % kTiles) * Tl::kBytes, bar = smem_u32(&sh.tiles[next % kTiles]);
                const int t0 = (int)((pt.first + next) * kC), values = p.V - v0 > 64 ? 2 : 1;
                mbar_arrive_expect_tx(bar, ((k ? KP / 64 : 0) + (q ? KP / 64 : 0) + (v ? values : 0)) * kPanelBytes);
                for (int j = 0; j < KP / 64; ++j) {
                    if (k)
                        tile_g2s(tile + Tl::K + 2 * j * kPanelBytes, &cp.map_k, 64 * j, t0, g, b, bar);
                    if (q)
                        tile_g2s(tile + Tl::Q + 2 * j * kPanelBytes, &cp.map_q, 64 * j, t0, g, b, bar);
                }
                for (int j = 0; v && j < values; ++j)
                    tile_g2s(tile + Tl::V + j * kPanelBytes, &cp.map_v, v0 + 64 * j, t0, h, b, bar);
            }
            __syncwarp();
        }
        if (!warp_wait(sh.prepared_free[i % kPrepareds], (uint32_t)(i / kPrepareds + 1) & 1))
            return;
        if (threadIdx.x % 32 == 0) {
            const uint32_t ready = smem_u32(&sh.prepared[i % kPrepareds]);
            const uint32_t bytes = p.y ? kForwardBytes : kStatesBytes;
            mbar_arrive_expect_tx(ready, bytes);
            bulk_g2s(smem_u32(tiles) + Tl::kAll + (uint32_t)(i % kPrepareds) * kPreparedBytes, cp.prepared + (pt.item * cp.chunks + pt.first + i) * cp.record,
                     bytes, ready);
        }
        __syncwarp();
    }
}

// The other loading warps: rows to operands.
template <int DT, int KP>
__device__ __forceinline__ void make_tiles(const ChunkParams &cp, ChunkShared &sh, uint8_t *tiles, const Part &pt, int64_t n)
{
    typedef Tile<KP> Tl;
    const DeltaParams &p = cp.d;
    const int thread = threadIdx.x - (kThreads - kLoadThreads), b = pt.item / p.H, h = pt.item % p.H, g = h / (p.H / p.G), v0 = pt.v0;
    const int64_t chunks = pt.chunks;
    for (int64_t i = 0; i < chunks; ++i) {
        const int64_t t0 = (pt.first + i) * kC;
        const int live = (int)(n - t0 < kC ? n - t0 : kC);
        uint8_t *tile = tiles + (i % kTiles) * Tl::kBytes;
        const float *f = reinterpret_cast<const float *>(tiles + Tl::kAll + (i % kPrepareds) * kPreparedBytes + kAtFactors);
        if (!warp_wait(sh.tiles[i % kTiles], (uint32_t)(i / kTiles) & 1) || !warp_wait(sh.prepared[i % kPrepareds], (uint32_t)(i / kPrepareds) & 1))
            break;
        make_panels<DT, KP>(tile + Tl::K, p.k + t0 * p.k_s[0] + b * p.k_s[1] + g * p.k_s[2], p.k_s[0], f + kFactorScaleK * kC, p.K, cp.vectors_k,
                            min(live, (int)f[kFactorEnd * kC + kEndGood]), thread);
        if (p.y) {
            make_panels<DT, KP>(tile + Tl::Q, p.q + t0 * p.q_s[0] + b * p.q_s[1] + g * p.q_s[2], p.q_s[0], f + kFactorScaleQ * kC, p.K, cp.vectors_q, live,
                                thread);
            if (thread < 2 * kC)
                sh.of_y[i & 3][thread] = f[kFactorQ * kC + thread];
        }
        if (live < kC || !cp.vectors_v || pt.unit || p.V - v0 < kRows)
            fill_values(tile + Tl::V, p.v + t0 * p.v_s[0] + b * p.v_s[1] + h * p.v_s[2] + v0, p.v_s[0], pt.unit ? 0 : p.V - v0, cp.vectors_v, live, thread);
        leave_out<DT>(tile + Tl::V, pt.unit ? 0 : p.V - v0, live, (int)t0, sh.bad, thread);
        shared_to_async();
        warp_arrive(sh.full[i % kTiles]);
    }
}

template <int DT, int KP>
__global__ void __launch_bounds__(kThreads, 1) mcc1d_delta_chunks_rows(const __grid_constant__ ChunkParams cp)
{
    extern __shared__ uint8_t raw_shared[];
    __shared__ ChunkShared sh;
    uint8_t *tiles = raw_shared + (1024 - smem_u32(raw_shared) % 1024) % 1024;
    const DeltaParams &p = cp.d;
    const int tid = threadIdx.x, warp = tid / 32, group = warp / 4;
    int64_t n;
    Part pt;
    if (!part_of(cp.seg, p, cp.tiles, p.state, p.final_state, pt, n))
        return;

    if (tid < kRows)
        sh.bad[tid] = INT_MAX;
    if (tid == 0) {
        sh.failed = 0;
        for (int i = 0; i < kTiles; ++i)
            mbar_init(smem_u32(&sh.tiles[i]), 1), mbar_init(smem_u32(&sh.full[i]), kLoadWarps), mbar_init(smem_u32(&sh.tile_free[i]), kRowWarps + 1);
        for (int i = 0; i < kPrepareds; ++i)
            mbar_init(smem_u32(&sh.prepared[i]), 1), mbar_init(smem_u32(&sh.prepared_free[i]), kRowWarps + 1);
        mbar_init(smem_u32(&sh.x), 1), mbar_init(smem_u32(&sh.u), 1), mbar_init(smem_u32(&sh.y), 1), mbar_init(smem_u32(&sh.end), 1);
        mbar_init(smem_u32(&sh.r), kRowWarps), mbar_init(smem_u32(&sh.v), kRowWarps), mbar_init(smem_u32(&sh.s), kRowWarps), mbar_init(smem_u32(&sh.out), 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kProductWarp)
        tmem_alloc(smem_u32(&sh.tmem), kColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();

    if (group < kParts) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegRows));
        hold_rows<DT, KP>(cp, sh, tiles, pt, n);
    } else if (group == kParts) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegY));
        if (p.y)
            write_y<DT>(cp, sh, pt, n);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegRest));
        if (warp > kCopyWarp)
            make_tiles<DT, KP>(cp, sh, tiles, pt, n);
        else if (warp == kCopyWarp)
            copy_tiles<KP>(cp, sh, tiles, pt);
        else if (tid % 32 == 0)
            issue_products<KP>(sh, smem_u32(tiles), pt.chunks, p.y != nullptr);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kProductWarp) {
        tmem_fence_after();
        tmem_free(sh.tmem, kColumns);
    }
    if (p.kept.u && tid < kRows && pt.v0 + tid < p.V) {
        const int64_t end = (pt.first + pt.chunks) * kC;
        for (int64_t t = sh.bad[tid]; t < n && t < end; ++t)
            p.kept.u[(t * p.B * p.H + pt.item) * p.kept.Vp + pt.v0 + tid] = __uint_as_float(0x7FFFFFFFu);
    }
}

template <int DT, int KP>
int32_t chunks_of(const ChunkParams &p, cudaStream_t stream)
{
    constexpr int bytes = Tile<KP>::kAll + kPrepareds * kPreparedBytes + 1024;
    // the rows' registers come out of what the block starts with: an increase
    // past that would wait for ever
    static const bool fits = [] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, mcc1d_delta_chunks_rows<DT, KP>) == cudaSuccess && fa.numRegs == kRegLaunch;
    }();
    if (!fits)
        return kErrCuda;
    if (cudaFuncSetAttribute(mcc1d_delta_chunks_rows<DT, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return kErrCuda;
    return launch(mcc1d_delta_chunks_rows<DT, KP>, dim3((unsigned)blocks_of(p.seg, p.d, p.tiles)), kThreads, bytes, stream, p);
}

}  // namespace

// Segments of the time axis: where heads are few, their chunks are shared out.
// A first pass takes every segment but the last from an empty state (the first
// from its own), and what becomes of any state on its way through it, K rows
// from the unit matrix; a join passes the states on; a second pass takes all
// segments at once. In units of a chunk's time, with waves of 152 blocks and two
// units for each join, the shortest division is taken, if it saves a fifth: 65536
// tokens of 6 heads of 64 take 3160 us in one piece and 418 us in 25 (241 + 36 + 141).
// Measured at that case only; a join of K = 128 reads four times as much.
static int64_t waves(int64_t blocks) { return (blocks + kNumSMs - 1) / kNumSMs; }

int32_t delta_segments(int64_t chunks, int64_t heads, int64_t tiles)
{
    int64_t best = 1, time = chunks * waves(heads * tiles) * 4 / 5;
    for (int64_t n = 2; n <= 64 && n * 2 <= chunks; ++n) {
        const int64_t per = (chunks + n - 1) / n;
        const int64_t t = per * (waves((n - 1) * heads * (tiles + 1)) + waves(n * heads * tiles)) + 2 * n;
        if (t < time)
            best = n, time = t;
    }
    return (int32_t)best;
}

// Prompts of less than half a chunk go token by token and take no workspace. 8
// sequences of 16 heads of 128 x 128 take 16 us so at 16 tokens and 30 at 31, and in a
// chunk 23 at any number up to 64; with gradients 56 and 81, and 63. The sides are even
// at about 22 tokens; 64 sequences take 35 us at 4 tokens and 166 at 31, where reading
// and writing the states would take 20.
DeltaPlan delta_plan(const mcc1d_delta_args &a, bool back)
{
    DeltaPlan p = {};
    p.chunks = (a.S + kChunk - 1) / kChunk;
    p.tokens = a.S < kChunk / 2;
    if (p.tokens)
        return p;
    const auto take = [&](uint64_t bytes) {
        const uint64_t at = p.bytes;
        p.bytes += (bytes + 255) / 256 * 256;
        return at;
    };
    p.off_prepared = take((uint64_t)(p.chunks * a.B * a.H) * (back ? kBothBytes : kForwardBytes));
    p.segments = delta_segments(p.chunks, a.B * a.H, (a.V + kRows - 1) / kRows);
    if (p.segments > 1) {
        const uint64_t joins = (uint64_t)(p.segments - 1) * a.B * a.H * a.K * 4;
        p.off_states = take(joins * a.V), p.off_turns = take(joins * a.K);
    }
    return p;
}

int32_t launch_delta_chunks(const mcc1d_delta_args &a, const DeltaPlan &plan, uint8_t *workspace, const DeltaKept &kept, cudaStream_t stream)
{
    ChunkParams p = {};
    p.d = delta_params(a);
    p.prepared = workspace + plan.off_prepared, p.record = kept.u ? kBothBytes : kForwardBytes;
    p.chunks = plan.chunks;
    p.tiles = (int32_t)((a.V + kRows - 1) / kRows);
    p.vectors_q = token_tiles(&p.map_q, a.q, a.S, a.B, a.G, a.K, a.q_strides, true);
    p.vectors_k = token_tiles(&p.map_k, a.k, a.S, a.B, a.G, a.K, a.k_strides, true);
    p.vectors_v = token_tiles(&p.map_v, a.v, a.S, a.B, a.H, a.V, a.v_strides, false);
    p.pairs_y = a.V % 2 == 0 && ((uintptr_t)a.y & 3u) == 0;
    p.vectors_s = a.K % 4 == 0 && ((uintptr_t)a.final_state & 15u) == 0;
    const auto go = [&]() {
        if (a.dtype == 0)
            return a.K <= 64 ? chunks_of<0, 64>(p, stream) : chunks_of<0, 128>(p, stream);
        return a.K <= 64 ? chunks_of<1, 64>(p, stream) : chunks_of<1, 128>(p, stream);
    };
    p.seg.count = plan.segments, p.seg.per = (plan.chunks + plan.segments - 1) / plan.segments;
    if (plan.segments > 1) {
        ChunkParams first = p;
        first.seg.states = reinterpret_cast<float *>(workspace + plan.off_states);
        first.seg.turns = reinterpret_cast<float *>(workspace + plan.off_turns);
        first.seg.ends = true;
        first.d.y = nullptr;
        first.vectors_s = a.K % 4 == 0;
        std::swap(p, first);
        int32_t st = go();
        std::swap(p, first);
        if (st == kOk)
            st = launch_delta_join(first.seg.states, first.seg.turns, a.B * a.H, (int32_t)a.V, (int32_t)a.K, plan.segments, false, stream);
        if (st != kOk)
            return st;
        p.seg.states = first.seg.states;
    }
    p.d.kept = kept;
    return go();
}

int32_t launch_delta(const mcc1d_delta_args &a, void *workspace, cudaStream_t stream)
{
    const DeltaPlan plan = delta_plan(a, false);
    if (plan.tokens)
        return launch_delta_tokens(a, DeltaKept(), stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const int32_t st = launch_delta_prepare(a, ws + plan.off_prepared, false, stream);
    return st == kOk ? launch_delta_chunks(a, plan, ws, DeltaKept(), stream) : st;
}

}  // namespace mcc1d
