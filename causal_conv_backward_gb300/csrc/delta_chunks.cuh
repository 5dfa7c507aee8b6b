// delta_chunks.cuh - what the gated delta rule's chunked passes share, forwards
// and backwards: the roles of a block's warps, rows of values on their way to
// operands, and bounds of rows.
#pragma once

#include "delta_common.cuh"
#include "tensor_core.cuh"
#include "tensor_map.h"

namespace mcc1d {

// 128 rows of a state, a row to four threads that share its columns; then four
// warps for what leaves by rows, one that issues products, one that copies
// tiles, and the ones that make operands of them.
constexpr int kC = kChunk, kRows = 128, kParts = 4;
constexpr int kRowWarps = 4 * kParts, kLoadWarps = 6, kLoadThreads = 32 * kLoadWarps, kThreads = 32 * (kRowWarps + 4 + 2 + kLoadWarps);
constexpr int kProductWarp = kRowWarps + 4, kCopyWarp = kProductWarp + 1;

// How the time axis is cut (delta_chunks.cu). With `ends` the pass is the one
// over all segments but the last, from empty states, that leaves `states` and,
// in a forward, `turns`; without, the segments begin with `states`.
struct Segments {
    int32_t count;            // 1: not at all
    int64_t per;              // chunks
    float *states, *turns;    // [count-1][heads][V,K], [count-1][heads][K,K]
    bool ends;
};
// A block's part: chunks, rows of V (or of the unit matrix), and where its rows'
// states come from and go to.
struct Part {
    int item, v0, rows;
    int64_t first, chunks;    // of its sequence
    const float *from;
    float *to;
    bool unit, last;
};
inline int64_t blocks_of(const Segments &g, const DeltaParams &p, int32_t tiles)
{
    const int64_t heads = (int64_t)p.B * p.H;
    return g.ends ? (g.count - 1) * heads * (tiles + (g.turns ? 1 : 0)) : g.count * heads * tiles;
}
// False where there is nothing to do.
__device__ __forceinline__ bool part_of(const Segments &g, const DeltaParams &p, int tiles, const float *state, float *final_state, Part &pt, int64_t &n)
{
    const int all = tiles + (g.ends && g.turns ? 1 : 0), heads = p.B * p.H;
    const int tile = blockIdx.x % all, segment = blockIdx.x / all / heads;
    pt.item = blockIdx.x / all % heads;
    pt.unit = tile == tiles;
    if (pt.unit && segment == 0)
        return false;
    n = clamped_length(p.lengths, pt.item / p.H, p.S);
    const int64_t chunks = (n + kChunk - 1) / kChunk;
    pt.first = segment * g.per < chunks ? segment * g.per : chunks;
    pt.chunks = chunks - pt.first < g.per ? chunks - pt.first : g.per;
    pt.v0 = pt.unit ? 0 : tile * kRows;
    pt.rows = pt.unit ? p.K : p.V;
    pt.last = segment == g.count - 1;
    const int64_t VK = (int64_t)p.V * p.K, KK = (int64_t)p.K * p.K, at = (int64_t)segment * heads + pt.item;
    pt.from = segment == 0 ? (state ? state + pt.item * VK : nullptr) : !g.ends ? g.states + (at - heads) * VK : nullptr;
    pt.to = pt.unit ? g.turns + at * KK : g.ends ? g.states + at * VK : pt.last && final_state ? final_state + pt.item * VK : nullptr;
    return true;
}

// The same backwards: the pass from empty gradients leaves out the first segment
// and puts the gradient that leaves segment j to states [j-1]; segment j of the
// other begins with states [j].
__device__ __forceinline__ void part_of_back(const Segments &g, const DeltaParams &p, int tiles, Part &pt, int64_t &n)
{
    const int heads = p.B * p.H, segment = blockIdx.x / tiles / heads + (g.ends ? 1 : 0);
    pt.item = blockIdx.x / tiles % heads;
    n = clamped_length(p.lengths, pt.item / p.H, p.S);
    const int64_t chunks = (n + kChunk - 1) / kChunk;
    pt.first = segment * g.per < chunks ? segment * g.per : chunks;
    pt.chunks = chunks - pt.first < g.per ? chunks - pt.first : g.per;
    pt.v0 = (blockIdx.x % tiles) * kRows;
    pt.rows = p.V;
    pt.unit = false;
    pt.last = segment == g.count - 1;
    const int64_t VK = (int64_t)p.V * p.K, at = (int64_t)segment * heads + pt.item;
    pt.from = pt.last ? (p.grad_final ? p.grad_final + pt.item * VK : nullptr) : g.ends ? nullptr : g.states + at * VK;
    pt.to = g.ends ? g.states + (at - heads) * VK : segment == 0 && p.grad_state ? p.grad_state + pt.item * VK : nullptr;
}

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

// Piece `piece` of a token's row: eight 16-bit values, from the copied rows in
// shared memory or, where they could not be copied, from global memory one by
// one; zeros behind the row's and the sequence's end.
__device__ __forceinline__ uint4 piece_of(const uint8_t *copied, const uint16_t *row, bool vectors, int live)
{
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (live > 0 && vectors)
        r = *reinterpret_cast<const uint4 *>(copied);
    if (live > 0 && !vectors) {
        uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live)
                w[i / 2] |= (uint32_t)__ldg(row + i) << (16 * (i % 2));
    }
    return r;
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

__device__ __forceinline__ void rows_meet() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kRowWarps) : "memory"); }
__device__ __forceinline__ float most_of_parts(const float (&x)[kParts][kRows], int r)
{
    static_assert(kParts == 4, "four parts of a row");
    return fmaxf(fmaxf(x[0][r], x[1][r]), fmaxf(x[2][r], x[3][r]));
}

// Values from `first` on of a row of n, times `of`, to memory.
template <int N>
__device__ __forceinline__ void write_row(float *row, int first, int n, bool vectors, const float (&s)[N], float of)
{
    row += first;
    if (vectors) {
#pragma unroll
        for (int k = 0; k < N; k += 4)
            if (first + k < n)
                *reinterpret_cast<float4 *>(row + k) = make_float4(s[k] * of, s[k + 1] * of, s[k + 2] * of, s[k + 3] * of);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (first + k < n)
                row[k] = s[k] * of;
    }
}

}  // namespace mcc1d
