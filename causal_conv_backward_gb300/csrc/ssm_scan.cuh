// ssm_scan.cuh - what the selective scan's forward and backward kernels share:
// their parameters, the tile loads and the sums over a channel's lanes.
//
// Layout of a block: NW recurrence warps; a channel's N states sit on NL lanes,
// four to a lane, and a lane holds them for K = 2 channels, so a warp owns
// 64/NL channels and the block CB = 64 NW/NL, of one group and one sequence. It
// walks one time chunk in tiles of TT rows. EW further warps do what is needed
// once per (row, channel): the loads, dt and the gate for the tile after the
// one the recurrence is in, and the outputs of the tile before it. A thread of
// theirs owns two adjacent channels of RP rows of the tile. The two kinds meet
// in shared memory, in two buffers, with one barrier per tile.
#pragma once

#include <atomic>

#include "device.h"
#include "ssm.h"
#include "ssm_common.cuh"

namespace mcc1d {

template <int NL_, int NW, int EW, int TT_>
struct ScanTile {
    static constexpr int NL = NL_, K = 2, TT = TT_, WARPS = NW;
    static constexpr int THREADS = 32 * (NW + EW), EL_THREADS = 32 * EW;
    static constexpr int NP = 4 * NL;              // states, padded
    static constexpr int CL = 32 / NL;             // lanes of one state
    static constexpr int CB = NW * CL * K;         // channels per block
    static constexpr int CP = CB / 2;              // channel pairs per row
    static constexpr int RG = EL_THREADS / CP;     // rows of one pass over a tile
    static constexpr int RP = TT / RG;             // rows per thread
    static_assert(RG >= 1 && RP >= 1 && RG * CP == EL_THREADS && RP * RG == TT, "a tile is whole passes");

    // A lane's number among a channel's NL, and its (first) channel / K in the
    // warp. Shared-memory loads of 8 and 16 bytes run at their full rate only
    // where lanes one apart, or two apart, read the same address (measured:
    // 2.1 against 4.0 cycles for 16 bytes): the states take lane bit 0 and the
    // bits above the channels', so that dt (same channel) repeats one apart
    // and B and C (same states) two apart.
    __device__ __forceinline__ static int state_lane(int lane)
    {
        return NL == 1 ? 0 : (lane & 1) | ((lane / (2 * CL)) << 1);
    }
    __device__ __forceinline__ static int channel_lane(int lane) { return NL == 1 ? lane : (lane >> 1) % CL; }
};

// Tiles of the forward. B and C are read from shared memory once for a lane's
// two channels, without which its bandwidth is the first limit (1024 tokens x 8
// sequences x 2048 channels: 107 us, with one channel per lane 124 us).
// At N = 16 the element warps are what a block alone on its SM waits for (222 us
// with or without the recurrence on 4096 x 1 x 2048), so they are four.
template <int NL>
using OutTile = ScanTile<NL, 2, (NL <= 4 ? 4 : NL == 8 ? 2 : 1), (NL == 1 ? 8 : 16)>;
// Tiles of the backward's first pass, with the rows and channels of its second.
template <int NL>
using BwdTile = ScanTile<NL, 4, (NL < 8 ? 4 : NL == 8 ? 2 : 1), (NL < 4 ? 4 * NL : 16)>;
// Tiles of the backward's second pass: the same rows and channels, and the
// recurrence warps do the elements' part too, so that every warp has the
// registers of a recurrence warp. Two channels per lane, so that grad_B's and
// grad_C's sums over channels start inside the lane.
template <int NL>
using BwdMainTile = ScanTile<NL, 4, 4, BwdTile<NL>::TT>;

struct ScanParams {
    const uint16_t *u, *delta, *z, *Bm, *Cm, *gy;
    const float *A, *D, *dbias, *h0, *gfs;
    const int32_t *lengths;
    uint16_t *y, *gu, *gdelta, *gz;
    float *hT, *gstate;
    float *e, *r, *dts, *cp, *cpdt, *ga, *gd, *bc;
    int64_t us, ub, ds, db, zs, zb, Bs, Bb, Bg, Cs, Cb, Cg, gs, gb;
    int64_t S, B, H, tiles, tiles_per_chunk, chunks;
    ScanGrid grid;                        // of the kernel launched
    int32_t N, G, Hg;
    int32_t softplus, pairs;              // pairs: every [S,B,H] row starts on 4 bytes and Hg is even
    int32_t bcpairs, bc8;                 // rows of B and C start on 4 (16) bytes and N is even (a multiple of 8)
    int32_t vecA, vecState;               // rows of A (of the states) can be moved 16 bytes at a time
};

int32_t launch_scan_bwd_main(const ScanParams &p, const ScanPlan &pl, const mcc1d_scan_bwd_args &a, cudaStream_t s);

// A kernel's shared-memory limit, raised once per context: a context created
// after a device reset starts without the attribute.
struct SharedReady {
    std::atomic<unsigned long long> ctx{0};
    bool set(const void *kernel, int bytes)
    {
        const unsigned long long now = current_context_id();
        if (now != 0 && ctx.load(std::memory_order_acquire) == now)
            return true;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return false;
        ctx.store(now != 0 ? now : current_context_id(), std::memory_order_release);
        return true;
    }
};

inline dim3 scan_launch_grid(const ScanParams &p)
{
    return dim3((unsigned)p.grid.blocks, (unsigned)p.B, (unsigned)p.chunks);
}

// Where a block works: blockIdx = (channel block, sequence, chunk).
struct ScanWhere {
    int64_t chunk, b;
    int32_t blk, g;
    int32_t c0;       // first channel
    int32_t nc;       // channels of the block inside the group
};

template <class T>
__device__ __forceinline__ ScanWhere scan_where(const ScanParams &p)
{
    ScanWhere w;
    w.blk = (int32_t)blockIdx.x;
    w.b = blockIdx.y;
    w.chunk = blockIdx.z;
    w.g = w.blk / p.grid.blocks_per_group;
    const int32_t in = (w.blk - w.g * p.grid.blocks_per_group) * T::CB;
    w.c0 = w.g * p.Hg + in;
    w.nc = p.Hg - in < T::CB ? p.Hg - in : T::CB;
    return w;
}

// Two adjacent 16-bit values, in one access (PAIRS: both are there) or two.
template <bool PAIRS>
__device__ __forceinline__ uint32_t load_pair(const uint16_t *p, bool one, bool two)
{
    if (PAIRS)
        return one ? __ldg(reinterpret_cast<const uint32_t *>(p)) : 0u;
    const uint32_t lo = one ? __ldg(p) : 0u, hi = two ? __ldg(p + 1) : 0u;
    return lo | (hi << 16);
}

template <bool PAIRS>
__device__ __forceinline__ void store_pair(uint16_t *p, uint32_t v, bool one, bool two)
{
    if (PAIRS) {
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

// Sums v[0..N-1] over L lanes, N and L powers of two. The lanes' numbers are
// made of the lane bits FIRST (the lowest), 2 REST, 4 REST and so on. Each
// exchange halves what a lane carries on, so N values cost N (1 - 1/L)
// shuffles where N >= L, not N log2 L. Lane number j is left with v[0..] = the
// sums of values j N/L .. (N >= L), or with v[0] = that of value j % N (N < L).
template <int N, int L, int FIRST, int REST>
__device__ __forceinline__ void lanes_sum(float (&v)[N], int lane)
{
    constexpr int M = N < L ? N : L;
    int n = N;
#pragma unroll
    for (int step = M / 2; step >= 1; step /= 2) {
        const int mask = step == 1 ? FIRST : step * REST;
        const bool up = (lane & mask) != 0;
        n /= 2;
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            if (i < n) {
                const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, mask);
            }
    }
#pragma unroll
    for (int step = M; step < L; step *= 2)
        v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], step == 1 ? FIRST : step * REST);
}

// The rows of B and C of one tile on their way to shared memory. Rows whose
// states start on 16 bytes and come in eights (p.bc8) move 16 bytes at a time,
// others a pair or one at a time. Rows from `rows` on are zeros, as are states
// past N. KC: C too, not B alone.
template <class T, bool KC>
struct BcTile {
    static constexpr int NP = T::NP, TT = T::TT, THREADS = T::EL_THREADS, TENSORS = KC ? 2 : 1;
    static constexpr int PAIRS = TENSORS * TT * NP / 2, WORDS = (PAIRS + THREADS - 1) / THREADS;
    static constexpr int EIGHTS = NP >= 8 ? PAIRS / 4 : 0, VECS = (EIGHTS + THREADS - 1) / THREADS;
    static constexpr int N = WORDS > 4 * VECS ? WORDS : 4 * VECS;
    uint32_t v[N];
    int id;                                  // of the thread, among THREADS
    const uint16_t *B_, *C_, *src[VECS > 0 ? VECS : 1];
    int64_t Bstep, Cstep;
    int row8[VECS > 0 ? VECS : 1];           // TT where there is nothing to load

    template <bool BOTH>
    __device__ __forceinline__ void load_pairs(const ScanParams &p, const uint16_t *B, const uint16_t *C, int rows)
    {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const int k = id + i * THREADS, q = k % (TT * NP / 2), row = q / (NP / 2), n = 2 * (q % (NP / 2));
            const bool on = k < PAIRS && row < rows, c = k >= TT * NP / 2;
            const uint16_t *src = c ? C + row * p.Cs + n : B + row * p.Bs + n;
            v[i] = load_pair<BOTH>(src, on && n < p.N, on && n + 1 < p.N);
        }
    }
    // The eight states of vector i: its tensor (C if true), row and first state.
    __device__ __forceinline__ bool place8(int i, int &row, int &n) const
    {
        const int k = id + i * THREADS, q = k % (EIGHTS / TENSORS);
        row = q / (NP / 8);
        n = 8 * (q % (NP / 8));
        return k >= EIGHTS / TENSORS;
    }
    // B, C: the first tile's first rows; dir: 1 where the tiles run forwards, -1 backwards.
    __device__ __forceinline__ void start(const ScanParams &p, const uint16_t *B, const uint16_t *C, int thread, int dir)
    {
        id = thread;
        B_ = B;
        C_ = C;
        Bstep = dir * TT * p.Bs;
        Cstep = dir * TT * p.Cs;
        if constexpr (VECS > 0) {
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                int row, n;
                const bool c = place8(i, row, n), in = id + i * THREADS < EIGHTS && n < p.N;
                src[i] = c ? C + row * p.Cs + n : B + row * p.Bs + n;
                row8[i] = in ? row : TT;
            }
        }
    }
    // The next tile, of which `rows` rows hold tokens.
    __device__ __forceinline__ void load(const ScanParams &p, int rows)
    {
        if constexpr (VECS > 0) {
            if (p.bc8) {
#pragma unroll
                for (int i = 0; i < VECS; ++i) {
                    uint4 r = make_uint4(0u, 0u, 0u, 0u);
                    if (row8[i] < rows)
                        r = __ldg(reinterpret_cast<const uint4 *>(src[i]));
                    src[i] += id + i * THREADS >= EIGHTS / TENSORS ? Cstep : Bstep;
                    v[4 * i] = r.x;
                    v[4 * i + 1] = r.y;
                    v[4 * i + 2] = r.z;
                    v[4 * i + 3] = r.w;
                }
                return;
            }
        }
        if (p.bcpairs)
            load_pairs<true>(p, B_, C_, rows);
        else
            load_pairs<false>(p, B_, C_, rows);
        B_ += Bstep;
        C_ += Cstep;
    }
    template <int DT>
    __device__ __forceinline__ void put(const ScanParams &p, float (*sB)[NP], float (*sC)[NP]) const
    {
        if constexpr (VECS > 0) {
            if (p.bc8) {
#pragma unroll
                for (int i = 0; i < VECS; ++i) {
                    int row, n;
                    const bool c = place8(i, row, n);
                    if (id + i * THREADS >= EIGHTS)
                        break;
                    float4 *dst = reinterpret_cast<float4 *>(KC && c ? &sC[row][n] : &sB[row][n]);
                    const float2 e = unpack2<DT>(v[4 * i]), f = unpack2<DT>(v[4 * i + 1]);
                    const float2 g = unpack2<DT>(v[4 * i + 2]), h = unpack2<DT>(v[4 * i + 3]);
                    dst[0] = make_float4(e.x, e.y, f.x, f.y);
                    dst[1] = make_float4(g.x, g.y, h.x, h.y);
                }
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const int k = id + i * THREADS, q = k % (TT * NP / 2), row = q / (NP / 2), n = 2 * (q % (NP / 2));
            if (k >= PAIRS)
                break;
            float *dst = KC && k >= TT * NP / 2 ? &sC[row][n] : &sB[row][n];
            *reinterpret_cast<float2 *>(dst) = unpack2<DT>(v[i]);
        }
    }
};

}  // namespace mcc1d
