// ssm_scan.cuh - what the selective scan's forward and backward kernels share:
// their parameters, the tile loads and the sums over a channel's lanes.
//
// Layout of a block: 8 warps; a channel's N states sit on NL lanes, four to a
// lane, so a warp owns 32/NL channels and the block CB = 256/NL, of one group
// and one sequence. It walks one time chunk in tiles of TT rows. Loads, dt and
// the gate are done once per (row, channel) by a thread that owns two adjacent
// channels of RP rows of the tile; dt and dt*u reach the lanes of the
// recurrence through shared memory, and y comes back the same way.
#pragma once

#include "ssm.h"
#include "ssm_common.cuh"

namespace mcc1d {

struct ScanParams;
int32_t launch_scan_bwd_main(const ScanParams &p, const ScanPlan &pl, const mcc1d_scan_bwd_args &a, cudaStream_t s);

constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;

template <int NL>
struct ScanTile {
    static constexpr int NP = 4 * NL;              // states, padded
    static constexpr int CW = 32 / NL;             // channels per warp
    static constexpr int CB = kScanWarps * CW;     // channels per block
    static constexpr int CP = CB / 2;              // channel pairs per row
    static constexpr int RG = kScanThreads / CP;   // rows of one pass over a tile
};

// Rows per tile: 2048 (row, channel) elements, at most 64 rows (forward) or 32
// (backward, whose shared memory per row is larger).
__host__ __device__ constexpr int scan_tile_rows(int nl, bool bwd) { return 8 * nl < (bwd ? 32 : 64) ? 8 * nl : (bwd ? 32 : 64); }

struct ScanParams {
    const uint16_t *u, *delta, *z, *Bm, *Cm, *gy;
    const float *A, *D, *dbias, *h0, *gfs;
    const int32_t *lengths;
    uint16_t *y, *gu, *gdelta, *gz;
    float *hT, *gstate;
    float *e, *r, *dts, *cp, *cpdt, *ga, *gd, *bc;
    int64_t us, ub, ds, db, zs, zb, Bs, Bb, Bg, Cs, Cb, Cg, gs, gb;
    int64_t S, B, H, blocks, tiles, tiles_per_chunk, chunks;
    int32_t N, G, Hg, blocks_per_group;
    int32_t softplus, pairs, bcpairs;     // pairs: every [S,B,H] row starts on 4 bytes and Hg is even
    int32_t vecA, vecState;               // rows of A (of the states) can be moved 16 bytes at a time
};

// Where a block works.
struct ScanWhere {
    int64_t chunk, b;
    int32_t blk, g;
    int32_t c0;       // first channel
    int32_t nc;       // channels of the block inside the group
};

template <int NL>
__device__ __forceinline__ ScanWhere scan_where(const ScanParams &p)
{
    ScanWhere w;
    const int64_t i = blockIdx.x;
    w.blk = (int32_t)(i % p.blocks);
    const int64_t q = i / p.blocks;
    w.b = q % p.B;
    w.chunk = q / p.B;
    w.g = w.blk / p.blocks_per_group;
    const int32_t in = (w.blk - w.g * p.blocks_per_group) * ScanTile<NL>::CB;
    w.c0 = w.g * p.Hg + in;
    w.nc = p.Hg - in < ScanTile<NL>::CB ? p.Hg - in : ScanTile<NL>::CB;
    return w;
}

// Two adjacent channels of one row (the second only where `two`).
__device__ __forceinline__ uint32_t load_pair(const uint16_t *p, bool one, bool two, bool wide)
{
    if (wide)
        return one ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
    const uint32_t lo = one ? __ldg(p) : 0u, hi = two ? __ldg(p + 1) : 0u;
    return lo | (hi << 16);
}

__device__ __forceinline__ void store_pair(uint16_t *p, uint32_t v, bool one, bool two, bool wide)
{
    if (wide) {
        if (one)
            *reinterpret_cast<uint32_t *>(p) = v;
        return;
    }
    if (one)
        p[0] = (uint16_t)v;
    if (two)
        p[1] = (uint16_t)(v >> 16);
}

// Four of a channel's N states, zeros past N.
__device__ __forceinline__ float4 load_states(const float *row, int n0, int N, bool vec)
{
    if (vec)
        return n0 < N ? *reinterpret_cast<const float4 *>(row + n0) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 v;
    v.x = n0 < N ? row[n0] : 0.f;
    v.y = n0 + 1 < N ? row[n0 + 1] : 0.f;
    v.z = n0 + 2 < N ? row[n0 + 2] : 0.f;
    v.w = n0 + 3 < N ? row[n0 + 3] : 0.f;
    return v;
}

__device__ __forceinline__ void store_states(float *row, int n0, int N, bool vec, float4 v)
{
    if (vec) {
        if (n0 < N)
            *reinterpret_cast<float4 *>(row + n0) = v;
        return;
    }
    if (n0 < N)
        row[n0] = v.x;
    if (n0 + 1 < N)
        row[n0 + 1] = v.y;
    if (n0 + 2 < N)
        row[n0 + 2] = v.z;
    if (n0 + 3 < N)
        row[n0 + 3] = v.w;
}

// softplus(x) = log(1 + e^x); past 20 it is x to fp32's last bit.
__device__ __forceinline__ float softplus(float x) { return x > 20.f ? x : log1pf(expf(x)); }

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

// The rows of B and C of one tile, as pairs of states.
template <int NL, int TT>
struct BcTile {
    static constexpr int NP = 4 * NL;
    static constexpr int TOTAL = TT * NP / 2;
    static constexpr int N = (TOTAL + kScanThreads - 1) / kScanThreads;
    uint32_t b[N], c[N];

    __device__ __forceinline__ void load(const ScanParams &p, const uint16_t *B, const uint16_t *C, int64_t t0,
                                         int64_t te)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = threadIdx.x + i * kScanThreads, row = k / (NP / 2), n = 2 * (k % (NP / 2));
            const bool on = k < TOTAL && t0 + row < te;
            b[i] = load_pair(B + (t0 + row) * p.Bs + n, on && n < p.N, on && n + 1 < p.N, p.bcpairs);
            c[i] = C ? load_pair(C + (t0 + row) * p.Cs + n, on && n < p.N, on && n + 1 < p.N, p.bcpairs) : 0u;
        }
    }
    template <int DT>
    __device__ __forceinline__ void put(float (*sB)[NP], float (*sC)[NP]) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = threadIdx.x + i * kScanThreads, row = k / (NP / 2), n = 2 * (k % (NP / 2));
            if (k < TOTAL) {
                *reinterpret_cast<float2 *>(&sB[row][n]) = unpack2<DT>(b[i]);
                if (sC)
                    *reinterpret_cast<float2 *>(&sC[row][n]) = unpack2<DT>(c[i]);
            }
        }
    }
};

}  // namespace mcc1d
