// delta_chunks_bwd.cu - the gradients of the gated delta rule's states, from
// the last chunk to the first, on the tensor cores.
//
// A block has up to 128 rows of one head's gradient G [V,K] of the state after
// the chunk, as delta_chunks.cu has the state. With the factors of
// delta_prepare.cu, T without the decays (which G's part passes all of, whatever
// token it goes through: none of its bits are lost where they are small), every chunk is
//   D0 = G K^T,  dU through the later tokens: dR = e^(c(end)-c) D0 T + grad_y (P T)    (tokens along the columns)
//   grad_v = b dR
//   G = e^c(end) G + grad_y^T (e^c Q) - (dR b e^c) K
// grad_y is exact in fp16 (each row's values scaled by a power of two, tokens that grow
// on their way to the end or fade by another: growth_of in delta_prepare.cu) and is
// multiplied from shared memory; e^c Q is two fp16 terms there. The chain is
// G - D0 - dR - G, and bounds the kernel; the products with grad_y run in its gaps.
// 2048 tokens of 8 x 16 heads of 128 x 128 take 205 us, 6.4 us a chunk, of which the
// operands of the two tiles that fit beside one another take most: grad_y with its
// rows' scales, e^c Q in two terms (one scale for all rows: 216 us with the same
// registers, 205 with 8 more for the warps that make operands). Warps 0 to 15 hold
// the rows, 16 to 19 write dR and grad_v, 20 issues the products, 21 copies the
// tiles, 22 to 27 make operands of them where they lie.
#include "delta_chunks.cuh"

namespace mcc1d {

namespace {

constexpr int kStages = 2;
// Registers by warpgroup: rows (four), the ones that write, and two for the rest.
constexpr int kRegRows = 72, kRegOut = 96, kRegRest = 56, kRegLaunch = 72;
static_assert(kParts * kRegRows + kRegOut + 2 * kRegRest <= kThreads / 128 * kRegLaunch && kRegRows == kRegLaunch, "what the block is launched with");

struct BackParams {
    CUtensorMap map_q, map_k, map_y;    // where rows can be copied as tiles
    DeltaParams d;
    const uint8_t *prepared;
    int64_t chunks;
    int32_t tiles;            // of 128 rows of V
    bool vectors_q, vectors_k, vectors_y, vectors_s;
    bool pairs_v;             // two rows of grad_v are one word
    Segments seg;
};

template <int KP>
struct Stage {
    static constexpr int kPanels = KP / 64 * kPanelBytes;
    static constexpr int K = 0, QHi = kPanels, QLo = 2 * kPanels, Y = 3 * kPanels, kPrepared = Y + kRows / 64 * kPanelBytes;
    static constexpr int kBytes = kPrepared + kBackBytes;
    static_assert(kBytes % 1024 == 0, "panels on 1024 bytes");
};

// Columns of tensor memory: sums, then operands (pairs of fp16). D0 and dR
// follow on one another and share theirs; G's update is summed over X and U.
enum { kX = 0, kU = 64, kYP = 128, kYQ = 192, kGHi = 320, kGLo = 384, kWHi = 448, kWLo = 480, kColumns = 512 };

struct BackShared {
    uint64_t full[kStages], empty[kStages], tiles[kStages], x, r, u, v, s, end, out;
    float of_u[2][kRows];                       // of the last two chunks: what a row's sums are multiplied by
    alignas(16) float of_out[4][3 * kC];                   // of the last four chunks: the factors of G's and of grad_y's part of dR, b
    alignas(16) float of_y[4][kRows], most_y[4][kRows];     // grad_y's factor (0 where there is none), and its largest, by rows
    float of_q[4];                              // Q's factor
    float most[kParts][kRows], sum_r[kParts][kRows];
    alignas(16) float most_of_warps[2][kLoadWarps][kRows];
    uint32_t tmem, failed;
};

// ------------------------------------------------------------------ the rows
template <int DT, int KP>
__device__ __forceinline__ void hold_rows(const BackParams &cp, BackShared &sh, const uint8_t *stages, const Part &pt)
{
    typedef Stage<KP> St;
    constexpr int HK = KP / kParts, HC = kC / kParts, UNIT = HK < 32 ? HK : 32;
    static_assert(HC == 16, "sixteen tokens to a thread");
    const DeltaParams &p = cp.d;
    const int warp = threadIdx.x / 32, r = threadIdx.x % kRows, part = warp / 4, row = pt.v0 + r;
    const int64_t BH = (int64_t)p.B * p.H, chunks = pt.chunks;
    const bool mine = row < p.V;
    const uint32_t lanes = sh.tmem + ((uint32_t)(32 * (warp % 4)) << 16);
    float s[HK];             // the gradient times `scale_s`, a power of two
    {
        const float *from = pt.from + (int64_t)row * p.K + part * HK;
#pragma unroll
        for (int k = 0; k < HK; ++k)
            s[k] = pt.from && mine && part * HK + k < p.K ? from[k] : 0.f;
    }
    // scales come from bounds, as in delta_chunks.cu
    sh.most[part][r] = most_of(s);
    rows_meet();
    float scale_s = scale_for(most_of_parts(sh.most, r));
    rows_meet();
#pragma unroll
    for (int k = 0; k < HK; ++k)
        s[k] *= scale_s;
    const uint32_t terms_s = lanes + kGHi + HK / 2 * part, terms_w = lanes + kWHi + HC / 2 * part;
    if (chunks > 0) {
#pragma unroll
        for (int c = 0; c < HK; c += UNIT)
            put_terms<UNIT>(s + c, terms_s + c / 2, terms_s + (kGLo - kGHi) + c / 2);
        terms_done(sh.s);
    }
    bool ok = true;          // no wait gave up
    for (int64_t i = 0;; ++i) {          // the chunks counted from the last
        const uint32_t parity = (uint32_t)(i & 1);
        if (!ok)
#pragma unroll
            for (int k = 0; k < HK; ++k)
                s[k] = __uint_as_float(0x7FFFFFFFu);
        if (i < chunks && mine && !cp.seg.ends) {
            const float of = inverse_scale(scale_s);
            float *to = p.kept.states + (((pt.first + chunks - 1 - i) * BH + pt.item) * p.K + part * HK) * p.kept.Vp + row;
#pragma unroll
            for (int k = 0; k < HK; ++k, to += p.kept.Vp)
                if (part * HK + k < p.K)
                    *to = s[k] * of;
        }
        if (i >= chunks) {
            if (pt.to && mine)
                write_row<HK>(pt.to + (int64_t)row * p.K, part * HK, p.K, cp.vectors_s, s, inverse_scale(scale_s));
            break;
        }
        const uint8_t *stage = stages + (i % kStages) * St::kBytes;
        const float *f = reinterpret_cast<const float *>(stage + St::kPrepared + kAtBackFactors), *ends = f + kFactorEnd * kC;
        f += part * HC;
        ok = warp_wait(sh.full[i % kStages], (uint32_t)(i / kStages) & 1);
        sh.most[part][r] = most_of(s);
        rows_meet();
        if (sh.failed) {         // all rows leave together; theirs are NaN
            ok = false;
            i = chunks - 1;
            continue;
        }
        const float of_s = inverse_scale(scale_s), most_s = most_of_parts(sh.most, r) * of_s;
        const float scale_u = scale_for(ends[kEndOfGrad] * most_s), of_u = inverse_scale(scale_u);
        const float scale_r = scale_for(fmaf(ends[kEndDuOfGrad], most_s, ends[kEndDuOfY] * sh.most_y[i & 3][r])), of_r = inverse_scale(scale_r);
        if (part == 0)
            sh.of_u[parity][r] = of_u;
        ok = ok && warp_wait(sh.x, parity);
        tmem_fence_after();
        uint32_t raw[HC];
        float x[HC];
        tmem_load(lanes + kX + HC * part, raw);
        tmem_wait(raw);
        {
            const float2 m = make_float2(of_s * scale_u, of_s * scale_u);
#pragma unroll
            for (int t = 0; t < HC; t += 2) {
                const float2 ft = *reinterpret_cast<const float2 *>(f + kFactorU * kC + t);
                const float2 a = mul2(mul2(ft, m), make_float2(__uint_as_float(raw[t]), __uint_as_float(raw[t + 1])));
                x[t] = a.x, x[t + 1] = a.y;
            }
        }
        put_terms<HC>(x, terms_w, terms_w + (kWLo - kWHi));
        terms_done(sh.r);
        ok = ok && warp_wait(sh.u, parity);
        tmem_fence_after();
        float2 sum = make_float2(0.f, 0.f);
        {
            uint32_t yp[HC];
            tmem_load(lanes + kU + HC * part, raw);
            tmem_load(lanes + kYP + HC * part, yp);
            tmem_wait(raw), tmem_wait(yp);
            const float2 mu = make_float2(-of_u * scale_r, -of_u * scale_r);
            const float of_y = -sh.of_y[i & 3][r] * scale_r;
            const float2 my = make_float2(of_y, of_y);
#pragma unroll
            for (int t = 0; t < HC; t += 2) {
                const float2 fg = *reinterpret_cast<const float2 *>(f + kFactorX * kC + t), fy = *reinterpret_cast<const float2 *>(f + kFactorXY * kC + t);
                const float2 a = fma2(mul2(fg, mu), make_float2(__uint_as_float(raw[t]), __uint_as_float(raw[t + 1])),
                                      mul2(mul2(fy, my), make_float2(__uint_as_float(yp[t]), __uint_as_float(yp[t + 1]))));
                sum = add2(sum, make_float2(fabsf(a.x), fabsf(a.y)));
                x[t] = a.x, x[t + 1] = a.y;
            }
        }
        sh.sum_r[part][r] = sum.x + sum.y;
        put_terms<HC>(x, terms_w, terms_w + (kWLo - kWHi));
        terms_done(sh.v);
        rows_meet();     // for sum_r, while the products run
        // |G| <= e^c(end) |G| + sum of |dR k| + 64 |grad_y| |q|, and no |k|, |q| is above 2^16 as an operand
        const float before = scale_s, end = ends[kEndDecay], of_q = sh.of_q[i & 3], of_yq = sh.of_y[i & 3][r] * of_q;
        scale_s = scale_for(fmaf(fabsf(end), most_s, ((sh.sum_r[0][r] + sh.sum_r[1][r]) + (sh.sum_r[2][r] + sh.sum_r[3][r])) * of_r * 65536.f) +
                            sh.most_y[i & 3][r] * (kC * 65536.f) * of_q);
        const float2 keep = make_float2(end * inverse_scale(before) * scale_s, end * inverse_scale(before) * scale_s);
        warp_arrive(sh.empty[i % kStages]);
        const float2 add = make_float2(of_r * scale_s, of_r * scale_s), add_y = make_float2(of_yq * scale_s, of_yq * scale_s);
        ok = ok && warp_wait(sh.end, parity);
        tmem_fence_after();
        if (!ok)
            sh.failed = 1;
#pragma unroll
        for (int c = 0; c < HK; c += 16) {
            uint32_t yq[16];
            tmem_load(lanes + kX + HK * part + c, raw);
            tmem_load(lanes + kYQ + HK * part + c, yq);
            tmem_wait(raw), tmem_wait(yq);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
                float2 o = fma2(add, make_float2(__uint_as_float(raw[k]), __uint_as_float(raw[k + 1])), mul2(keep, make_float2(s[c + k], s[c + k + 1])));
                o = fma2(add_y, make_float2(__uint_as_float(yq[k]), __uint_as_float(yq[k + 1])), o);
                s[c + k] = o.x, s[c + k + 1] = o.y;
            }
            if (i + 1 < chunks)
                put_terms<16>(s + c, terms_s + c / 2, terms_s + (kGLo - kGHi) + c / 2);
        }
        if (i + 1 < chunks)
            terms_done(sh.s);
    }
}

// ------------------------------------------------------------------ dR and grad_v
template <int DT>
__device__ __forceinline__ void write_rows(const BackParams &cp, BackShared &sh, const Part &pt, int64_t n)
{
    const DeltaParams &p = cp.d;
    const int r = threadIdx.x % kRows, row = pt.v0 + r;
    const int64_t BH = (int64_t)p.B * p.H, step = BH * p.V, step_u = BH * p.kept.Vp, chunks = pt.chunks, item = pt.item;
    const bool mine = row < p.V, odd = r & 1;
    const uint32_t lanes = sh.tmem + ((uint32_t)(32 * (threadIdx.x / 32 % 4)) << 16);
    // tokens of no chunk
    uint16_t *to = p.grad_v + (int64_t)item * p.V + row;
    if (mine && pt.last)
        for (int64_t t = (pt.first + chunks) * kC; t < p.S; ++t)
            to[t * step] = 0;
    int64_t i = 0;
    for (; i < chunks; ++i) {
        if (!warp_wait(sh.u, (uint32_t)(i & 1)))
            break;
        tmem_fence_after();
        const int64_t t0 = (pt.first + chunks - 1 - i) * kC;
        const float of_u = sh.of_u[i & 1][r], of_y = sh.of_y[i & 3][r];
        const float *fg = sh.of_out[i & 3], *fy = fg + kC, *bt = fy + kC;
        const int live = (int)(n - t0 < kC ? n - t0 : kC), rows = (int)(p.S - t0 < kC ? p.S - t0 : kC);
        const bool whole = cp.pairs_v && rows == kC && live == kC;
        uint32_t dr[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t y[16];
            tmem_load(lanes + kU + 16 * c, dr[c]);
            tmem_load(lanes + kYP + 16 * c, y);
            tmem_wait(dr[c]), tmem_wait(y);
#pragma unroll
            for (int t = 0; t < 16; t += 2) {
                const float2 g = *reinterpret_cast<const float2 *>(fg + 16 * c + t), f = *reinterpret_cast<const float2 *>(fy + 16 * c + t);
                const float2 a = fma2(mul2(g, make_float2(of_u, of_u)), make_float2(__uint_as_float(dr[c][t]), __uint_as_float(dr[c][t + 1])),
                                      mul2(mul2(f, make_float2(of_y, of_y)), make_float2(__uint_as_float(y[t]), __uint_as_float(y[t + 1]))));
                dr[c][t] = __float_as_uint(a.x), dr[c][t + 1] = __float_as_uint(a.y);
            }
        }
        tmem_fence_before();
        warp_arrive(sh.out);
        float *to_u = p.kept.u + (t0 * BH + item) * p.kept.Vp + row;
        uint16_t *at = to + t0 * step, *pair = odd ? at + step - 1 : at;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (whole) {
#pragma unroll
                for (int t = 0; t < 16; t += 2, to_u += 2 * step_u, pair += 2 * step) {
                    const float a = __uint_as_float(dr[c][t]), e = __uint_as_float(dr[c][t + 1]);
                    if (mine)
                        to_u[0] = a, to_u[step_u] = e;
                    const uint32_t both = pack2<DT>(mul2(make_float2(a, e), *reinterpret_cast<const float2 *>(bt + 16 * c + t)));
                    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, both, 1);
                    if (mine)       // two rows of one token: even lanes the first, odd lanes the second
                        *reinterpret_cast<uint32_t *>(pair) = odd ? __byte_perm(other, both, 0x7632) : __byte_perm(both, other, 0x5410);
                }
            } else {
#pragma unroll
                for (int t = 0; t < 16; ++t, to_u += step_u, at += step) {
                    const float a = __uint_as_float(dr[c][t]);
                    const bool there = 16 * c + t < live;
                    if (mine && there)
                        *to_u = a;
                    if (mine && 16 * c + t < rows)
                        *at = there ? (uint16_t)pack2<DT>(make_float2(a * bt[16 * c + t], 0.f)) : (uint16_t)0;
                }
            }
        }
    }
    if (mine && i < chunks)         // a wait gave up
        for (int64_t t = pt.first * kC; t < (pt.first + chunks - i) * kC && t < p.S; ++t)
            to[t * step] = 0x7FFF;
}

// ------------------------------------------------------------------ products
// Second terms first, as in delta_chunks.cu.
template <int KP>
__device__ __forceinline__ void issue_products(BackShared &sh, uint32_t stages, int64_t chunks, bool out)
{
    typedef Stage<KP> St;
    constexpr uint32_t by_rows = mma_kind(kC, false), by_columns = mma_kind(KP, true), tokens_by_columns = mma_kind(kC, true);
    constexpr uint32_t y_tokens = mma_kind(kC, true, true), y_keys = mma_kind(KP, true, true);
    const uint32_t tmem = sh.tmem;
    const auto wait = [](uint64_t &bar, uint32_t parity) { return mbar_wait_bounded_inline(smem_u32(&bar), parity); };
    for (int64_t i = 0; i < chunks; ++i) {
        const uint32_t parity = (uint32_t)(i & 1), stage = stages + (uint32_t)(i % kStages) * St::kBytes;
        if (!wait(sh.full[i % kStages], (uint32_t)(i / kStages) & 1) || !wait(sh.s, parity))
            break;
        tmem_fence_after();
#pragma unroll
        for (int j = 0; j < KP / 16; ++j)
            mma_ts(tmem + kX, tmem + kGLo + 8 * j, desc_rows(stage + St::K + (j / 4) * kPanelBytes) + 2 * (j % 4), by_rows, j > 0);
#pragma unroll
        for (int j = 0; j < KP / 16; ++j)
            mma_ts(tmem + kX, tmem + kGHi + 8 * j, desc_rows(stage + St::K + (j / 4) * kPanelBytes) + 2 * (j % 4), by_rows, true);
        mma_commit(smem_u32(&sh.x));
        constexpr uint64_t step = 2048 >> 4;                // sixteen rows
        const uint64_t y = desc_columns(stage + St::Y, kPanelBytes);
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ss(tmem + kYP, y + step * j, desc_columns(stage + St::kPrepared + kAtBackPTLo, kPanelBytes) + step * j, y_tokens, j > 0);
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ss(tmem + kYP, y + step * j, desc_columns(stage + St::kPrepared + kAtBackPT, kPanelBytes) + step * j, y_tokens, true);
        if (!wait(sh.r, parity))
            break;
        tmem_fence_after();
#pragma unroll
        for (int j = 0; j < kC / 16; ++j) {
            mma_ts(tmem + kU, tmem + kWHi + 8 * j, desc_columns(stage + St::kPrepared + kAtBackTLo, kPanelBytes) + step * j, tokens_by_columns, j > 0);
            mma_ts(tmem + kU, tmem + kWLo + 8 * j, desc_columns(stage + St::kPrepared + kAtBackT, kPanelBytes) + step * j, tokens_by_columns, true);
        }
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ts(tmem + kU, tmem + kWHi + 8 * j, desc_columns(stage + St::kPrepared + kAtBackT, kPanelBytes) + step * j, tokens_by_columns, true);
        mma_commit(smem_u32(&sh.u));
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ss(tmem + kYQ, y + step * j, desc_columns(stage + St::QLo, kPanelBytes) + step * j, y_keys, j > 0);
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ss(tmem + kYQ, y + step * j, desc_columns(stage + St::QHi, kPanelBytes) + step * j, y_keys, true);
        if (!wait(sh.v, parity) || (out && !wait(sh.out, parity)))
            break;
        tmem_fence_after();
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ts(tmem + kX, tmem + kWLo + 8 * j, desc_columns(stage + St::K, kPanelBytes) + step * j, by_columns, j > 0);
#pragma unroll
        for (int j = 0; j < kC / 16; ++j)
            mma_ts(tmem + kX, tmem + kWHi + 8 * j, desc_columns(stage + St::K, kPanelBytes) + step * j, by_columns, true);
        mma_commit(smem_u32(&sh.end));
        mma_commit(smem_u32(&sh.empty[i % kStages]));
    }
}

// ------------------------------------------------------------------ tiles
template <int KP>
__device__ __forceinline__ void copy_tiles(const BackParams &cp, BackShared &sh, uint8_t *stages, const Part &pt)
{
    typedef Stage<KP> St;
    const DeltaParams &p = cp.d;
    const int b = pt.item / p.H, h = pt.item % p.H, g = h / (p.H / p.G), v0 = pt.v0;
    const int64_t chunks = pt.chunks;
    const bool k = cp.vectors_k, q = cp.vectors_q, y = cp.vectors_y;
    for (int64_t i = 0; i < chunks; ++i) {
        if (!warp_wait(sh.empty[i % kStages], (uint32_t)(i / kStages + 1) & 1))
            break;
        if (threadIdx.x % 32 == 0) {
            const int64_t chunk = pt.first + chunks - 1 - i;
            const uint32_t stage = smem_u32(stages) + (uint32_t)(i % kStages) * St::kBytes, bar = smem_u32(&sh.tiles[i % kStages]);
            const int t0 = (int)(chunk * kC), values = p.V - v0 > 64 ? 2 : 1;
            mbar_arrive_expect_tx(bar, kBackBytes + ((k ? KP / 64 : 0) + (q ? KP / 64 : 0) + (y ? values : 0)) * kPanelBytes);
            bulk_g2s(stage + St::kPrepared, cp.prepared + (pt.item * cp.chunks + chunk) * kBothBytes + kStatesBytes, kBackBytes, bar);
            for (int j = 0; j < KP / 64; ++j) {
                if (k)
                    tile_g2s(stage + St::K + j * kPanelBytes, &cp.map_k, 64 * j, t0, g, b, bar);
                if (q)
                    tile_g2s(stage + St::QHi + j * kPanelBytes, &cp.map_q, 64 * j, t0, g, b, bar);
            }
            for (int j = 0; y && j < values; ++j)
                tile_g2s(stage + St::Y + j * kPanelBytes, &cp.map_y, v0 + 64 * j, t0, h, b, bar);
        }
        __syncwarp();
    }
}

__device__ __forceinline__ uint4 scaled_half(const float2 (&x)[4], float by)
{
    const float2 f = make_float2(by, by);
    return make_uint4(pack_half2(mul2(x[0], f)), pack_half2(mul2(x[1], f)), pack_half2(mul2(x[2], f)), pack_half2(mul2(x[3], f)));
}
template <int DT>
__device__ __forceinline__ void unpack8(const uint4 &v, float2 (&x)[4])
{
    x[0] = unpack2<DT>(v.x), x[1] = unpack2<DT>(v.y), x[2] = unpack2<DT>(v.z), x[3] = unpack2<DT>(v.w);
}

template <int DT, int KP>
__device__ __forceinline__ void make_tiles(const BackParams &cp, BackShared &sh, uint8_t *stages, const Part &pt, int64_t n)
{
    typedef Stage<KP> St;
    const DeltaParams &p = cp.d;
    const int thread = threadIdx.x - (kThreads - kLoadThreads), b = pt.item / p.H, h = pt.item % p.H, g = h / (p.H / p.G), v0 = pt.v0;
    const int64_t chunks = pt.chunks;
    for (int64_t i = 0; i < chunks; ++i) {
        const int64_t t0 = (pt.first + chunks - 1 - i) * kC;
        const int live = (int)(n - t0 < kC ? n - t0 : kC);
        uint8_t *stage = stages + (i % kStages) * St::kBytes;
        const float *f = reinterpret_cast<const float *>(stage + St::kPrepared + kAtBackFactors);
        if (!warp_wait(sh.tiles[i % kStages], (uint32_t)(i / kStages) & 1))
            break;
        // grad_y: the largest value of each row first; a thread has eight rows of every STEP_Yth token
        constexpr int PIECES_Y = kRows / 8, STEP_Y = kLoadThreads / PIECES_Y, PIECES = KP / 8, STEP = kLoadThreads / PIECES;
        static_assert(PIECES_Y == 16, "two lanes of a warp to the same rows");
        const uint16_t *gy = p.grad_y + t0 * p.gy_s[0] + b * p.gy_s[1] + h * p.gy_s[2] + v0;
        const int piece_y = thread % PIECES_Y, live_y = p.V - v0 - 8 * piece_y;
        uint8_t *panel_y = stage + St::Y + (piece_y / 8) * kPanelBytes;
        float2 scale[4];
        {
            float2 most[4] = {};
#pragma unroll 1
            for (int t = thread / PIECES_Y; t < kC; t += STEP_Y) {
                float2 x[4];
                unpack8<DT>(piece_of(panel_y + panel_at(t, piece_y % 8), gy + t * p.gy_s[0] + 8 * piece_y, cp.vectors_y, t < live ? live_y : 0), x);
                const float2 by = make_float2(f[kFactorY * kC + t], f[kFactorY * kC + t]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = mul2(x[e], by);
                    most[e] = make_float2(fmaxf(most[e].x, fabsf(x[e].x)), fmaxf(most[e].y, fabsf(x[e].y)));
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                most[e] = make_float2(fmaxf(most[e].x, __shfl_xor_sync(0xFFFFFFFFu, most[e].x, 16)), fmaxf(most[e].y, __shfl_xor_sync(0xFFFFFFFFu, most[e].y, 16)));
            float4 *to = reinterpret_cast<float4 *>(&sh.most_of_warps[i & 1][thread / 32][8 * piece_y]);
            if (thread % 32 < 16)
                to[0] = make_float4(most[0].x, most[0].y, most[1].x, most[1].y), to[1] = make_float4(most[2].x, most[2].y, most[3].x, most[3].y);
            asm volatile("bar.sync 2, %0;" ::"n"(kLoadThreads) : "memory");
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kLoadWarps; ++w) {
                    const float4 o = reinterpret_cast<const float4 *>(&sh.most_of_warps[i & 1][w][8 * piece_y])[half];
                    m = make_float4(fmaxf(m.x, o.x), fmaxf(m.y, o.y), fmaxf(m.z, o.z), fmaxf(m.w, o.w));
                }
                // times a token's factor, and still a number
                const auto of = [](float most) { return fminf(scale_for(most), 0x1p100f); };
                scale[2 * half] = make_float2(of(m.x), of(m.y)), scale[2 * half + 1] = make_float2(of(m.z), of(m.w));
                if (thread < PIECES_Y) {
                    const auto back = [](float most, float scale) { return most == 0.f ? 0.f : inverse_scale(scale); };
                    reinterpret_cast<float4 *>(&sh.most_y[i & 3][8 * piece_y])[half] = m;
                    reinterpret_cast<float4 *>(&sh.of_y[i & 3][8 * piece_y])[half] =
                        make_float4(back(m.x, scale[2 * half].x), back(m.y, scale[2 * half].y), back(m.z, scale[2 * half + 1].x), back(m.w, scale[2 * half + 1].y));
                }
            }
        }
        const float scale_q = scale_for(f[kFactorEnd * kC + kEndMostQ] * 32768.f);       // rows of q are below 2^15 as operands
        if (thread == 0)
            sh.of_q[i & 3] = inverse_scale(scale_q);
        if (thread < 3 * kC)
            sh.of_out[i & 3][thread] = f[(thread < kC ? kFactorT : thread < 2 * kC ? kFactorP : kFactorB) * kC + thread % kC];
#pragma unroll 1
        for (int t = thread / PIECES_Y; t < kC; t += STEP_Y) {
            uint8_t *at = panel_y + panel_at(t, piece_y % 8);
            float2 x[4];
            unpack8<DT>(piece_of(at, gy + t * p.gy_s[0] + 8 * piece_y, cp.vectors_y, t < live ? live_y : 0), x);
            const float2 by = make_float2(f[kFactorY * kC + t], f[kFactorY * kC + t]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = mul2(x[e], mul2(scale[e], by));
            *reinterpret_cast<uint4 *>(at) = make_uint4(pack_half2(x[0]), pack_half2(x[1]), pack_half2(x[2]), pack_half2(x[3]));
        }
        const int piece = thread % PIECES, live_k = p.K - 8 * piece;
        const uint16_t *k = p.k + t0 * p.k_s[0] + b * p.k_s[1] + g * p.k_s[2] + 8 * piece, *q = p.q + t0 * p.q_s[0] + b * p.q_s[1] + g * p.q_s[2] + 8 * piece;
        const int panel = (piece / 8) * kPanelBytes;
#pragma unroll 1
        for (int t = thread / PIECES; t < kC; t += STEP) {
            const uint32_t off = panel + panel_at(t, piece % 8);
            float2 x[4];
            unpack8<DT>(piece_of(stage + St::K + off, k + t * p.k_s[0], cp.vectors_k, t < live ? live_k : 0), x);
            *reinterpret_cast<uint4 *>(stage + St::K + off) = scaled_half(x, f[kFactorScaleK * kC + t]);
            unpack8<DT>(piece_of(stage + St::QHi + off, q + t * p.q_s[0], cp.vectors_q, t < live ? live_k : 0), x);
            const float by = f[kFactorScaleQ * kC + t], of = f[kFactorQ * kC + t] * scale_q;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                two_terms(mul2(mul2(x[e], make_float2(by, by)), make_float2(of, of)), hi[e], lo[e]);
            *reinterpret_cast<uint4 *>(stage + St::QHi + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(stage + St::QLo + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        shared_to_async();
        warp_arrive(sh.full[i % kStages]);
    }
}

template <int DT, int KP>
__global__ void __launch_bounds__(kThreads, 1) mcc1d_delta_chunks_bwd_rows(const __grid_constant__ BackParams cp)
{
    extern __shared__ uint8_t raw_shared[];
    __shared__ BackShared sh;
    uint8_t *stages = raw_shared + (1024 - smem_u32(raw_shared) % 1024) % 1024;
    const DeltaParams &p = cp.d;
    const int tid = threadIdx.x, warp = tid / 32, group = warp / 4;
    int64_t n;
    Part pt;
    part_of_back(cp.seg, p, cp.tiles, pt, n);

    if (tid == 0) {
        sh.failed = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), kLoadWarps);
            mbar_init(smem_u32(&sh.empty[i]), kRowWarps + 1);
            mbar_init(smem_u32(&sh.tiles[i]), 1);
        }
        mbar_init(smem_u32(&sh.x), 1), mbar_init(smem_u32(&sh.u), 1), mbar_init(smem_u32(&sh.end), 1);
        mbar_init(smem_u32(&sh.r), kRowWarps), mbar_init(smem_u32(&sh.v), kRowWarps), mbar_init(smem_u32(&sh.s), kRowWarps);
        mbar_init(smem_u32(&sh.out), 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kProductWarp)
        tmem_alloc(smem_u32(&sh.tmem), kColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();

    if (group < kParts) {
        hold_rows<DT, KP>(cp, sh, stages, pt);
    } else if (group == kParts) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegOut));
        if (!cp.seg.ends)
            write_rows<DT>(cp, sh, pt, n);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegRest));
        if (warp > kCopyWarp)
            make_tiles<DT, KP>(cp, sh, stages, pt, n);
        else if (warp == kCopyWarp)
            copy_tiles<KP>(cp, sh, stages, pt);
        else if (tid % 32 == 0)
            issue_products<KP>(sh, smem_u32(stages), pt.chunks, !cp.seg.ends);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == kProductWarp) {
        tmem_fence_after();
        tmem_free(sh.tmem, kColumns);
    }
}

template <int DT, int KP>
int32_t chunks_of(const BackParams &p, cudaStream_t stream)
{
    constexpr int bytes = kStages * Stage<KP>::kBytes + 1024;
    // the registers of the warps that write come out of what the block starts
    // with: an increase past that would wait for ever
    static const bool fits = [] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, mcc1d_delta_chunks_bwd_rows<DT, KP>) == cudaSuccess && fa.numRegs == kRegLaunch;
    }();
    if (!fits)
        return kErrCuda;
    if (cudaFuncSetAttribute(mcc1d_delta_chunks_bwd_rows<DT, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return kErrCuda;
    return launch(mcc1d_delta_chunks_bwd_rows<DT, KP>, dim3((unsigned)blocks_of(p.seg, p.d, p.tiles)), kThreads, bytes, stream, p);
}

}  // namespace

int32_t launch_delta_chunks_bwd(const mcc1d_delta_bwd_args &a, const DeltaPlan &plan, const uint8_t *forward, float *grads, const DeltaKept &kept,
                                cudaStream_t stream)
{
    const mcc1d_delta_args &f = a.fwd;
    BackParams p = {};
    p.d = delta_params(f);
    p.d.kept = kept;
    p.d.grad_y = static_cast<const uint16_t *>(a.grad_y), p.d.grad_v = static_cast<uint16_t *>(a.grad_v);
    p.d.grad_final = a.grad_final_state, p.d.grad_state = a.grad_state;
    for (int i = 0; i < 3; ++i)
        p.d.gy_s[i] = a.grad_y_strides[i];
    p.prepared = forward + plan.off_prepared;
    p.chunks = plan.chunks;
    p.tiles = (int32_t)((f.V + kRows - 1) / kRows);
    p.vectors_q = token_tiles(&p.map_q, f.q, f.S, f.B, f.G, f.K, f.q_strides, true);
    p.vectors_k = token_tiles(&p.map_k, f.k, f.S, f.B, f.G, f.K, f.k_strides, true);
    p.vectors_y = token_tiles(&p.map_y, a.grad_y, f.S, f.B, f.H, f.V, a.grad_y_strides, true);
    p.vectors_s = f.K % 4 == 0 && ((uintptr_t)a.grad_state & 15u) == 0;
    p.pairs_v = f.V % 2 == 0 && ((uintptr_t)a.grad_v & 3u) == 0;
    p.seg.count = plan.segments, p.seg.per = (plan.chunks + plan.segments - 1) / plan.segments;
    const auto go = [&]() {
        if (f.dtype == 0)
            return f.K <= 64 ? chunks_of<0, 64>(p, stream) : chunks_of<0, 128>(p, stream);
        return f.K <= 64 ? chunks_of<1, 64>(p, stream) : chunks_of<1, 128>(p, stream);
    };
    if (plan.segments > 1) {
        p.seg.states = grads;
        p.seg.ends = true;
        const bool vectors = p.vectors_s;
        p.vectors_s = f.K % 4 == 0;
        int32_t st = go();
        if (st == kOk)
            st = launch_delta_join(grads, reinterpret_cast<const float *>(forward + plan.off_turns), f.B * f.H, (int32_t)f.V, (int32_t)f.K, plan.segments, true,
                                   stream);
        if (st != kOk)
            return st;
        p.seg.ends = false;
        p.vectors_s = vectors;
    }
    return go();
}

}  // namespace mcc1d
