// delta_chunks.cu - the gated delta rule over prompts, a chunk of 64 tokens at
// a time, on the tensor cores.
//
// A block has one head's state [V,K], up to 128 rows of it, a row to two
// threads that share its columns: everything that goes along a row (decays,
// sums, scales, rounding to two fp16 terms) stays in them, and the state itself
// in their registers, in fp32. With the factors of delta_prepare.cu, a chunk is
//   X = S K^T        R = b V - e^c X          (A: the state, from tensor memory)
//   U = R T^T        Y = e^c S Q^T + R (PT)^T
//   S = e^c(end) S + (U e^(c(end)-c)) K
// with tokens along the columns. Operands in tensor memory are two fp16 terms of
// fp32 rows scaled by a power of two, 22 bits; K and Q are exact in fp16 (rows
// scaled by a power of two), so those products take two terms and those
// with T and P T three. Sums are fp32.
//
// The chunks of one head follow on one another, X - R - U - S, and bound the
// kernel: the products' latency and the conversions between them, for which a
// scheduler has two warps of rows. Y is taken in the gaps and leaves through
// warps of its own. Warps 0 to 7 hold the rows, 8 to 11 write Y, 12 issues the
// products, 13 to 15 bring the next chunk's tiles.
#include "delta_common.cuh"
#include "tensor_core.cuh"

namespace mcc1d {

namespace {

constexpr int kC = kChunk, kRows = 128, kLoadThreads = 96, kThreads = 512, kStages = 2;
// Registers by warpgroup: rows, rows, Y, the rest; together what the block has.
constexpr int kRegRows = 168, kRegY = 96, kRegRest = 80;
static_assert(2 * kRegRows + kRegY + kRegRest == 4 * 128, "65536 registers");

struct ChunkParams {
    DeltaParams d;
    const uint8_t *prepared;
    int64_t chunks;
    int32_t tiles;            // of 128 rows of V
    bool vectors_q, vectors_k, vectors_v, vectors_s;
    bool pairs_y;             // two rows of y are one word
};

template <int KP>
struct Stage {
    static constexpr int kPanels = KP / 64 * kPanelBytes;
    static constexpr int K = 0, Q = kPanels, kPrepared = 2 * kPanels;
    static constexpr int V = kPrepared + (kChunkBytes + 1023) / 1024 * 1024;      // [token pair][row] of two values
    static constexpr int kBytes = V + kC * kRows * 2;
    static_assert(kBytes % 1024 == 0, "panels on 1024 bytes");
};

// Columns of tensor memory: sums, then operands (pairs of fp16).
enum { kX = 0, kU = 64, kQS = 128, kPR = 192, kSHi = 256, kSLo = 320, kRHi = 384, kRLo = 416, kUHi = 448, kULo = 480, kColumns = 512 };

struct ChunkShared {
    uint64_t full[kStages], empty[kStages], factors[kStages], x, r, u, v, y, s, end, out;
    float of_s[2][kRows], of_r[2][kRows];       // of the last two chunks: what rows' terms are multiplied by
    float most[2][kRows], most_v[2][kRows], sum_u[2][kRows];      // of the halves of a row
    uint32_t tmem, failed;
};

// A wait of a whole warp; false where it gave up.
__device__ __forceinline__ bool warp_wait(uint64_t &bar, uint32_t parity)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait_bounded_inline(smem_u32(&bar), parity));
}
__device__ __forceinline__ void warp_arrive(uint64_t &bar)
{
    __syncwarp();
    if (threadIdx.x % 32 == 0)
        mbar_arrive(smem_u32(&bar));
}

// Eight 16-bit values to shared memory, `live` of them from global memory and
// zeros behind: as an asynchronous copy where addresses allow 16 bytes.
template <bool VECTORS>
__device__ __forceinline__ void bring_eight(uint32_t to, const uint16_t *from, int live)
{
    if constexpr (VECTORS) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live > 0 ? 16 : 0) : "memory");
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = i < live ? __ldg(from + i) : 0u;
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(w[0] | w[1] << 16), "r"(w[2] | w[3] << 16), "r"(w[4] | w[5] << 16),
                     "r"(w[6] | w[7] << 16)
                     : "memory");
    }
}

// A chunk's rows of q or k on their way to panels. A loading thread has one
// piece of every STEPth row, so that little is left to compute per piece.
template <int KP, bool VECTORS>
__device__ __forceinline__ void bring_rows(uint32_t panels, const uint16_t *from, int64_t step, int K, int n, int thread)
{
    constexpr int PIECES = KP / 8, STEP = kLoadThreads / PIECES;
    static_assert(kLoadThreads % PIECES == 0, "whole rows");
    const int piece = thread % PIECES, live = K - 8 * piece;
    int t = thread / PIECES;
    panels += (piece / 8) * kPanelBytes;
    const uint16_t *row = from + t * step + 8 * piece;
#pragma unroll 2
    for (; t < kC; t += STEP, row += STEP * step) {
        const bool there = t < n && live > 0;
        bring_eight<VECTORS>(panels + panel_at(t, piece % 8), there ? row : from, there ? live : 0);
    }
}
// Pieces made scaled fp16 where they are, by the thread that brought them.
template <int DT, int KP>
__device__ __forceinline__ void make_half(uint8_t *panels, const float *scales, int thread)
{
    constexpr int PIECES = KP / 8, STEP = kLoadThreads / PIECES, N = (kC + STEP - 1) / STEP, BATCH = 4;
    const int piece = thread % PIECES, t0 = thread / PIECES;
    panels += (piece / 8) * kPanelBytes;
#pragma unroll
    for (int j = 0; j < N; j += BATCH) {
        uint4 v[BATCH];
        float s[BATCH];
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
            const int t = t0 + (j + e) * STEP;
            if (t < kC)
                v[e] = *reinterpret_cast<const uint4 *>(panels + panel_at(t, piece % 8)), s[e] = scales[t];
        }
#pragma unroll
        for (int e = 0; e < BATCH; ++e) {
            const int t = t0 + (j + e) * STEP;
            const float2 f = make_float2(s[e], s[e]);
            if (t < kC)
                *reinterpret_cast<uint4 *>(panels + panel_at(t, piece % 8)) =
                    make_uint4(pack_half2(mul2(unpack2<DT>(v[e].x), f)), pack_half2(mul2(unpack2<DT>(v[e].y), f)),
                               pack_half2(mul2(unpack2<DT>(v[e].z), f)), pack_half2(mul2(unpack2<DT>(v[e].w), f)));
        }
    }
}

// A chunk's rows of v: pieces of two tokens side by side, then exchanged to
// pairs of tokens by the thread that brought them.
constexpr int kPiecesV = kRows / 8, kStepV = kLoadThreads / kPiecesV;
template <bool VECTORS>
__device__ __forceinline__ void bring_values(uint32_t to, const uint16_t *from, int64_t step, int V, int n, int thread)
{
    const int piece = thread % kPiecesV, live = V - 8 * piece;
    int t = 2 * (thread / kPiecesV);
    to += 32 * thread;
    const uint16_t *row = from + t * step + 8 * piece;
#pragma unroll 2
    for (; t < kC; t += 2 * kStepV, row += 2 * kStepV * step, to += 32 * kLoadThreads) {
        const bool one = t < n && live > 0, two = t + 1 < n && live > 0;
        bring_eight<VECTORS>(to, one ? row : from, one ? live : 0);
        bring_eight<VECTORS>(to + 16, two ? row + step : from, two ? live : 0);
    }
}
__device__ __forceinline__ void pair_values(uint8_t *v, int thread)
{
#pragma unroll 3
    for (int e = thread; e < kC / 2 * kPiecesV; e += kLoadThreads) {
        uint4 *at = reinterpret_cast<uint4 *>(v + 32 * e);
        const uint4 x = at[0], y = at[1];
        at[0] = make_uint4(__byte_perm(x.x, y.x, 0x5410), __byte_perm(x.x, y.x, 0x7632), __byte_perm(x.y, y.y, 0x5410), __byte_perm(x.y, y.y, 0x7632));
        at[1] = make_uint4(__byte_perm(x.z, y.z, 0x5410), __byte_perm(x.z, y.z, 0x7632), __byte_perm(x.w, y.w, 0x5410), __byte_perm(x.w, y.w, 0x7632));
    }
}

// Scaled values of a row as terms in N / 2 columns from `hi` and `lo` on.
template <int N>
__device__ __forceinline__ void put_terms(const float *x, uint32_t hi, uint32_t lo)
{
    uint32_t h[N / 2], l[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e)
        two_terms(make_float2(x[2 * e], x[2 * e + 1]), h[e], l[e]);
    tmem_store(hi, h);
    tmem_store(lo, l);
}
// What is stored is there for the products that are issued after an arrival.
__device__ __forceinline__ void terms_done(uint64_t &bar)
{
    tmem_wait_stores();
    tmem_fence_before();
    warp_arrive(bar);
}

template <int N>
__device__ __forceinline__ float most_of(const float (&x)[N])
{
    float m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < N; ++i)
        m[i % 4] = fmaxf(m[i % 4], fabsf(x[i]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// ------------------------------------------------------------------ the rows
template <int DT, int KP>
__device__ __forceinline__ void hold_rows(const ChunkParams &cp, ChunkShared &sh, const uint8_t *stages, int item, int b, int v0, int64_t n,
                                          int64_t chunks)
{
    typedef Stage<KP> St;
    constexpr int HK = KP / 2, HC = kC / 2;
    const DeltaParams &p = cp.d;
    const int warp = threadIdx.x / 32, r = threadIdx.x % kRows, half = warp / 4, row = v0 + r;
    const int64_t BH = (int64_t)p.B * p.H, VK = (int64_t)p.V * p.K;
    const bool mine = row < p.V;
    const uint32_t lanes = sh.tmem + ((uint32_t)(32 * (warp % 4)) << 16);
    float s[HK];             // the state times `scale_s`, a power of two
    {
        const float *from = p.state + item * VK + (int64_t)row * p.K + half * HK;
#pragma unroll
        for (int k = 0; k < HK; ++k)
            s[k] = p.state && mine && half * HK + k < p.K ? from[k] : 0.f;
    }
    float scale_s;
    // Scales come from bounds, so that no thread waits for its row's other half
    // where the products wait for it: terms keep 22 bits of a row up to 2^17 below
    // its bound. The state's largest value is known a phase late, the sum of a
    // row's |U| in time.
    sh.most[half][r] = most_of(s);
    asm volatile("bar.sync 1, 256;" ::: "memory");
    scale_s = scale_for(fmaxf(sh.most[0][r], sh.most[1][r]));
    asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
    for (int k = 0; k < HK; ++k)
        s[k] *= scale_s;
    const uint32_t terms_s = lanes + kSHi + HK / 2 * half, terms_r = lanes + kRHi + HC / 2 * half, terms_u = lanes + kUHi + HC / 2 * half;
    if (chunks > 0) {
        sh.of_s[0][r] = inverse_scale(scale_s);
#pragma unroll
        for (int c = 0; c < HK; c += 32)
            put_terms<32>(s + c, terms_s + c / 2, terms_s + (kSLo - kSHi) + c / 2);
        terms_done(sh.s);
    }
    bool ok = true;          // no wait gave up
    for (int64_t i = 0;; ++i) {
        const uint32_t parity = (uint32_t)(i & 1);
        if (!ok)
#pragma unroll
            for (int k = 0; k < HK; ++k)
                s[k] = __uint_as_float(0x7FFFFFFFu);
        float *to = i == chunks ? (p.final_state ? p.final_state + item * VK : nullptr) : p.states ? p.states + (i * BH + item) * VK : nullptr;
        if (to && mine) {
            const float of = inverse_scale(scale_s);
            to += (int64_t)row * p.K + half * HK;
            if (cp.vectors_s) {
#pragma unroll
                for (int k = 0; k < HK; k += 4)
                    if (half * HK + k < p.K)
                        *reinterpret_cast<float4 *>(to + k) = make_float4(s[k] * of, s[k + 1] * of, s[k + 2] * of, s[k + 3] * of);
            } else {
#pragma unroll
                for (int k = 0; k < HK; ++k)
                    if (half * HK + k < p.K)
                        to[k] = s[k] * of;
            }
        }
        if (i >= chunks)
            break;
        const uint8_t *stage = stages + (i % kStages) * St::kBytes;
        const float *f = reinterpret_cast<const float *>(stage + St::kPrepared + 4 * kPanelBytes), *ends = f + kFactorEnd * kC;
        const uint32_t *v = reinterpret_cast<const uint32_t *>(stage + St::V) + half * (HC / 2) * kRows + r;
        f += half * HC;
        // the products wait for the chunk's tiles too, but this thread reads some itself
        ok = warp_wait(sh.full[i % kStages], (uint32_t)(i / kStages) & 1);
        float most_v = 0.f;
#pragma unroll 4
        for (int t = 0; t < HC / 2; ++t) {
            const float2 x = unpack2<DT>(v[t * kRows]);
            most_v = fmaxf(most_v, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
        sh.most[half][r] = most_of(s);
        sh.most_v[half][r] = most_v;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (sh.failed) {         // all rows leave together; theirs are NaN
            ok = false;
            i = chunks - 1;
            continue;
        }
        const float of_s = inverse_scale(scale_s), most_s = fmaxf(sh.most[0][r], sh.most[1][r]) * of_s;
        const float bound_r = fmaf(ends[kEndOfV], fmaxf(sh.most_v[0][r], sh.most_v[1][r]), ends[kEndOfState] * most_s);
        const float scale_r = scale_for(bound_r), of_r = inverse_scale(scale_r);
        const float scale_u = scale_for(bound_r * ends[kEndOfR]), of_u = inverse_scale(scale_u), end = ends[kEndDecay];
        if (half == 0)
            sh.of_r[parity][r] = of_r;
        ok = ok && warp_wait(sh.x, parity);
        tmem_fence_after();
        const float2 mx = make_float2(-of_s * scale_r, -of_s * scale_r), mv = make_float2(scale_r, scale_r);
#pragma unroll 1
        for (int t0 = 0; t0 < HC; t0 += 16) {
            uint32_t raw[16];
            float x[16];
            tmem_load(lanes + kX + HC * half + t0, raw);
            tmem_wait(raw);
#pragma unroll
            for (int t = 0; t < 16; t += 2) {
                const float2 bt = *reinterpret_cast<const float2 *>(f + kFactorB * kC + t0 + t), ft = *reinterpret_cast<const float2 *>(f + kFactorX * kC + t0 + t);
                const float2 a = fma2(mul2(ft, mx), make_float2(__uint_as_float(raw[t]), __uint_as_float(raw[t + 1])),
                                      mul2(mul2(bt, mv), unpack2<DT>(v[(t0 + t) / 2 * kRows])));
                x[t] = a.x, x[t + 1] = a.y;
            }
            put_terms<16>(x, terms_r + t0 / 2, terms_r + (kRLo - kRHi) + t0 / 2);
        }
        terms_done(sh.r);
        ok = ok && warp_wait(sh.u, parity);
        tmem_fence_after();
        float2 sum_u = make_float2(0.f, 0.f);
        const float2 mu = make_float2(of_r * scale_u, of_r * scale_u);
#pragma unroll 1
        for (int t0 = 0; t0 < HC; t0 += 16) {
            uint32_t raw[16];
            float x[16];
            tmem_load(lanes + kU + HC * half + t0, raw);
            tmem_wait(raw);
            if (p.u && mine) {
                const int64_t at = i * kC + half * HC + t0, step = BH * p.V;
                float *to_u = p.u + (at * BH + item) * p.V + row;
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
            put_terms<16>(x, terms_u + t0 / 2, terms_u + (kULo - kUHi) + t0 / 2);
        }
        sh.sum_u[half][r] = sum_u.x + sum_u.y;
        terms_done(sh.v);
        warp_arrive(sh.empty[i % kStages]);
        asm volatile("bar.sync 1, 256;" ::: "memory");     // for sum_u, while the products run
        // |S| <= e^c(end) |S| + sum of |U k|, and no |k| is above 2^16 as an operand
        const float before = scale_s;
        scale_s = scale_for(fmaf(fabsf(end), most_s, (sh.sum_u[0][r] + sh.sum_u[1][r]) * of_u * 65536.f));
        const float2 keep = make_float2(end * inverse_scale(before) * scale_s, end * inverse_scale(before) * scale_s);
        const float2 add = make_float2(of_u * scale_s, of_u * scale_s);
        if (half == 0)
            sh.of_s[parity ^ 1][r] = inverse_scale(scale_s);
        ok = ok && warp_wait(sh.end, parity);
        tmem_fence_after();
        if (!ok)
            sh.failed = 1;
#pragma unroll
        for (int c = 0; c < HK; c += 32) {
            uint32_t raw[32];
            tmem_load(lanes + kX + HK * half + c, raw);
            tmem_wait(raw);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
                const float2 o = fma2(add, make_float2(__uint_as_float(raw[k]), __uint_as_float(raw[k + 1])), mul2(keep, make_float2(s[c + k], s[c + k + 1])));
                s[c + k] = o.x, s[c + k + 1] = o.y;
            }
            if (i + 1 < chunks)
                put_terms<32>(s + c, terms_s + c / 2, terms_s + (kSLo - kSHi) + c / 2);
        }
        if (i + 1 < chunks)
            terms_done(sh.s);
    }
}

// ------------------------------------------------------------------ Y
template <int DT, int KP>
__device__ __forceinline__ void write_y(const ChunkParams &cp, ChunkShared &sh, const uint8_t *stages, int item, int v0, int64_t n, int64_t chunks)
{
    typedef Stage<KP> St;
    const DeltaParams &p = cp.d;
    const int r = threadIdx.x % kRows, row = v0 + r;
    const int64_t step = (int64_t)p.B * p.H * p.V;
    const bool mine = row < p.V;
    const uint32_t lanes = sh.tmem + ((uint32_t)(32 * (threadIdx.x / 32 % 4)) << 16);
    uint16_t *to = p.y + (int64_t)item * p.V + row;
    const bool odd = r & 1;
    uint16_t *pair = odd ? to + step - 1 : to;
    int64_t i = 0;
    for (; i < chunks; ++i) {
        const uint8_t *stage = stages + (i % kStages) * St::kBytes;
        const float *f = reinterpret_cast<const float *>(stage + St::kPrepared + 4 * kPanelBytes);
        if (!warp_wait(sh.full[i % kStages], (uint32_t)(i / kStages) & 1) || !warp_wait(sh.y, (uint32_t)(i & 1)))
            break;
        tmem_fence_after();
        const float2 of_s = make_float2(sh.of_s[i & 1][r], sh.of_s[i & 1][r]), of_r = make_float2(sh.of_r[i & 1][r], sh.of_r[i & 1][r]);
        const int live = (int)(n - i * kC < kC ? n - i * kC : kC), rows = (int)(p.S - i * kC < kC ? p.S - i * kC : kC);
        const bool whole = cp.pairs_y && rows == kC && live == kC;
#pragma unroll 1
        for (int t0 = 0; t0 < kC; t0 += 8) {
            uint32_t a[8], c[8];
            tmem_load(lanes + kQS + t0, a);
            tmem_load(lanes + kPR + t0, c);
            tmem_wait(a), tmem_wait(c);
#pragma unroll
            for (int t = 0; t < 8; t += 2) {
                const int at = t0 + t;
                const float2 fq = *reinterpret_cast<const float2 *>(f + kFactorQ * kC + at), fp = *reinterpret_cast<const float2 *>(f + kFactorP * kC + at);
                const float2 y = fma2(mul2(fp, of_r), make_float2(__uint_as_float(c[t]), __uint_as_float(c[t + 1])),
                                      mul2(mul2(fq, of_s), make_float2(__uint_as_float(a[t]), __uint_as_float(a[t + 1]))));
                const uint32_t both = pack2<DT>(y);
                if (whole) {        // two rows of one token: even lanes the first, odd lanes the second
                    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, both, 1);
                    if (mine)
                        *reinterpret_cast<uint32_t *>(pair) = odd ? __byte_perm(other, both, 0x7632) : __byte_perm(both, other, 0x5410);
                } else {
                    if (mine && at < rows)
                        to[0] = at < live ? (uint16_t)both : (uint16_t)0;
                    if (mine && at + 1 < rows)
                        to[step] = at + 1 < live ? (uint16_t)(both >> 16) : (uint16_t)0;
                }
                to += 2 * step, pair += 2 * step;
            }
        }
        tmem_fence_before();
        warp_arrive(sh.out);
        warp_arrive(sh.empty[i % kStages]);
    }
    if (mine)
        for (int64_t t = i * kC; t < p.S; ++t, to += step)
            *to = i < chunks ? 0x7FFF : 0;          // NaN where a wait gave up
}

// ------------------------------------------------------------------ products
// One thread's. `y`: those of Y too.
template <int KP>
__device__ __forceinline__ void issue_products(ChunkShared &sh, uint32_t stages, int64_t chunks, bool y)
{
    typedef Stage<KP> St;
    constexpr uint32_t by_rows = mma_kind(kC, false), by_columns = mma_kind(KP, true);
    const uint32_t tmem = sh.tmem;
    const auto with_state = [&](uint32_t d, uint32_t panels) {
#pragma unroll
        for (int j = 0; j < KP / 16; ++j) {
            const uint64_t k = desc_rows(panels + (j / 4) * kPanelBytes) + 2 * (j % 4);
            mma_ts(tmem + d, tmem + kSHi + 8 * j, k, by_rows, j > 0);
            mma_ts(tmem + d, tmem + kSLo + 8 * j, k, by_rows, true);
        }
    };
    const auto with_r = [&](uint32_t d, uint32_t panels) {
#pragma unroll
        for (int j = 0; j < kC / 16; ++j) {
            const uint64_t hi = desc_rows(panels) + 2 * j, lo = desc_rows(panels + kPanelBytes) + 2 * j;
            mma_ts(tmem + d, tmem + kRHi + 8 * j, hi, by_rows, j > 0);
            mma_ts(tmem + d, tmem + kRHi + 8 * j, lo, by_rows, true);
            mma_ts(tmem + d, tmem + kRLo + 8 * j, hi, by_rows, true);
        }
    };
    const auto wait = [](uint64_t &bar, uint32_t parity) { return mbar_wait_bounded_inline(smem_u32(&bar), parity); };
    for (int64_t i = 0; i < chunks; ++i) {
        const uint32_t parity = (uint32_t)(i & 1), stage = stages + (uint32_t)(i % kStages) * St::kBytes;
        if (!wait(sh.full[i % kStages], (uint32_t)(i / kStages) & 1) || !wait(sh.s, parity))
            break;
        tmem_fence_after();
        with_state(kX, stage + St::K);
        mma_commit(smem_u32(&sh.x));
        if (!wait(sh.r, parity))
            break;
        tmem_fence_after();
        with_r(kU, stage + St::kPrepared);
        mma_commit(smem_u32(&sh.u));
        if (y) {
            if (!wait(sh.out, parity ^ 1))         // the Y before this one has been read
                break;
            tmem_fence_after();
            with_state(kQS, stage + St::Q);
            with_r(kPR, stage + St::kPrepared + 2 * kPanelBytes);
            mma_commit(smem_u32(&sh.y));
        }
        if (!wait(sh.v, parity))
            break;
        tmem_fence_after();
#pragma unroll
        for (int j = 0; j < kC / 16; ++j) {
            const uint64_t k = desc_columns(stage + St::K, kPanelBytes) + (uint64_t)(2048 * j >> 4);
            mma_ts(tmem + kX, tmem + kUHi + 8 * j, k, by_columns, j > 0);
            mma_ts(tmem + kX, tmem + kULo + 8 * j, k, by_columns, true);
        }
        mma_commit(smem_u32(&sh.end));
        mma_commit(smem_u32(&sh.empty[i % kStages]));
    }
}

// ------------------------------------------------------------------ tiles
template <int DT, int KP>
__device__ __forceinline__ void bring_tiles(const ChunkParams &cp, ChunkShared &sh, uint8_t *stages, int item, int b, int h, int v0, int64_t n,
                                            int64_t chunks)
{
    typedef Stage<KP> St;
    const DeltaParams &p = cp.d;
    const int thread = threadIdx.x - (kThreads - kLoadThreads), g = h / (p.H / p.G);
    for (int64_t i = 0; i < chunks; ++i) {
        const int64_t t0 = i * kC;
        const int live = (int)(n - t0 < kC ? n - t0 : kC);
        uint8_t *stage = stages + (i % kStages) * St::kBytes;
        if (!warp_wait(sh.empty[i % kStages], (uint32_t)(i / kStages + 1) & 1))
            break;
        if (thread == 0) {
            const uint32_t bar = smem_u32(&sh.factors[i % kStages]);
            mbar_arrive_expect_tx(bar, kChunkBytes);
            bulk_g2s(smem_u32(stage + St::kPrepared), cp.prepared + (item * cp.chunks + i) * kChunkBytes, kChunkBytes, bar);
        }
        const uint16_t *k = p.k + t0 * p.k_s[0] + b * p.k_s[1] + g * p.k_s[2], *q = p.q + t0 * p.q_s[0] + b * p.q_s[1] + g * p.q_s[2];
        const uint16_t *v = p.v + t0 * p.v_s[0] + b * p.v_s[1] + h * p.v_s[2] + v0;
        const uint32_t at = smem_u32(stage);
        if (cp.vectors_k)
            bring_rows<KP, true>(at + St::K, k, p.k_s[0], p.K, live, thread);
        else
            bring_rows<KP, false>(at + St::K, k, p.k_s[0], p.K, live, thread);
        if (cp.vectors_v)
            bring_values<true>(at + St::V, v, p.v_s[0], p.V - v0, live, thread);
        else
            bring_values<false>(at + St::V, v, p.v_s[0], p.V - v0, live, thread);
        if (!p.y) {
        } else if (cp.vectors_q)
            bring_rows<KP, true>(at + St::Q, q, p.q_s[0], p.K, live, thread);
        else
            bring_rows<KP, false>(at + St::Q, q, p.q_s[0], p.K, live, thread);
        asm volatile("cp.async.wait_all;" ::: "memory");
        pair_values(stage + St::V, thread);
        if (!warp_wait(sh.factors[i % kStages], (uint32_t)(i / kStages) & 1))
            break;
        const float *f = reinterpret_cast<const float *>(stage + St::kPrepared + 4 * kPanelBytes);
        make_half<DT, KP>(stage + St::K, f + kFactorScaleK * kC, thread);
        if (p.y)
            make_half<DT, KP>(stage + St::Q, f + kFactorScaleQ * kC, thread);
        shared_to_async();
        warp_arrive(sh.full[i % kStages]);
    }
}

template <int DT, int KP>
__global__ void __launch_bounds__(kThreads, 1) delta_chunks_kernel(const __grid_constant__ ChunkParams cp)
{
    extern __shared__ uint8_t raw_shared[];
    __shared__ ChunkShared sh;
    uint8_t *stages = raw_shared + (1024 - smem_u32(raw_shared) % 1024) % 1024;
    const DeltaParams &p = cp.d;
    const int tid = threadIdx.x, warp = tid / 32, group = warp / 4;
    const int item = blockIdx.x / cp.tiles, v0 = (blockIdx.x % cp.tiles) * kRows, b = item / p.H, h = item % p.H;
    const int64_t n = clamped_length(p.lengths, b, p.S), chunks = (n + kC - 1) / kC;

    if (tid == 0) {
        sh.failed = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), kLoadThreads / 32);
            mbar_init(smem_u32(&sh.empty[i]), 8 + (p.y ? 4 : 0) + 1);
            mbar_init(smem_u32(&sh.factors[i]), 1);
        }
        mbar_init(smem_u32(&sh.x), 1), mbar_init(smem_u32(&sh.u), 1), mbar_init(smem_u32(&sh.y), 1), mbar_init(smem_u32(&sh.end), 1);
        mbar_init(smem_u32(&sh.r), 8), mbar_init(smem_u32(&sh.v), 8), mbar_init(smem_u32(&sh.s), 8), mbar_init(smem_u32(&sh.out), 4);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12)
        tmem_alloc(smem_u32(&sh.tmem), kColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();

    if (group < 2) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegRows));
        hold_rows<DT, KP>(cp, sh, stages, item, b, v0, n, chunks);
    } else if (group == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegY));
        if (p.y)
            write_y<DT, KP>(cp, sh, stages, item, v0, n, chunks);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegRest));
        if (warp > 12)
            bring_tiles<DT, KP>(cp, sh, stages, item, b, h, v0, n, chunks);
        else if (tid % 32 == 0)
            issue_products<KP>(sh, smem_u32(stages), chunks, p.y != nullptr);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 12) {
        tmem_fence_after();
        tmem_free(sh.tmem, kColumns);
    }
}

template <int DT, int KP>
int32_t chunks_of(const ChunkParams &p, cudaStream_t stream)
{
    constexpr int bytes = kStages * Stage<KP>::kBytes + 1024;
    if (cudaFuncSetAttribute(delta_chunks_kernel<DT, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return kErrCuda;
    return launch(delta_chunks_kernel<DT, KP>, dim3((unsigned)((int64_t)p.d.B * p.d.H * p.tiles)), kThreads, bytes, stream, p);
}

}  // namespace

DeltaPlan delta_plan(const mcc1d_delta_args &a)
{
    DeltaPlan p = {};
    p.chunks = (a.S + kChunk - 1) / kChunk;
    p.tokens = a.S < 32;
    p.bytes = p.tokens ? 0 : (uint64_t)(p.chunks * a.B * a.H) * kChunkBytes;
    return p;
}

int32_t launch_delta_chunks(const mcc1d_delta_args &a, const uint8_t *prepared, cudaStream_t stream)
{
    ChunkParams p = {};
    p.d = delta_params(a);
    p.prepared = prepared;
    p.chunks = (a.S + kChunk - 1) / kChunk;
    p.tiles = (int32_t)((a.V + kRows - 1) / kRows);
    const auto vectors = [](int64_t n, const void *at, const int64_t (&s)[3]) { return vectors_for(n, (uintptr_t)at, s[0] | s[1] | s[2]); };
    p.vectors_q = vectors(a.K, a.q, a.q_strides), p.vectors_k = vectors(a.K, a.k, a.k_strides), p.vectors_v = vectors(a.V, a.v, a.v_strides);
    p.pairs_y = a.V % 2 == 0 && ((uintptr_t)a.y & 3u) == 0;
    p.vectors_s = a.K % 4 == 0 && ((uintptr_t)a.final_state & 15u) == 0;
    if (a.dtype == 0)
        return a.K <= 64 ? chunks_of<0, 64>(p, stream) : chunks_of<0, 128>(p, stream);
    return a.K <= 64 ? chunks_of<1, 64>(p, stream) : chunks_of<1, 128>(p, stream);
}

int32_t launch_delta(const mcc1d_delta_args &a, void *workspace, cudaStream_t stream)
{
    if (delta_plan(a).tokens)
        return launch_delta_tokens(a, nullptr, nullptr, stream);
    uint8_t *prepared = static_cast<uint8_t *>(workspace);
    const int32_t st = launch_delta_prepare(a, prepared, stream);
    return st == kOk ? launch_delta_chunks(a, prepared, stream) : st;
}

}  // namespace mcc1d
