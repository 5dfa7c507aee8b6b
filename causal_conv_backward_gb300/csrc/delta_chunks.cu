// delta_chunks.cu - the gated delta rule over prompts, a chunk of 64 tokens at
// a time, on the tensor cores.
//
// A block has one head's state [V,K], up to 128 rows of it, a row to a thread:
// everything that goes along a row (decays, sums, scales, rounding to two fp16
// terms) stays in the thread, and the state itself in its registers, in fp32.
// With the factors of delta_prepare.cu, every chunk is
//   X = S K^T        R = b V - e^c X          (A: the state, from tensor memory)
//   U = R T^T        Y = e^c S Q^T + R (PT)^T
//   S = e^c(end) S + (U e^(c(end)-c)) K
// with tokens along the columns. Operands in tensor memory are two fp16 terms of
// fp32 rows scaled by a power of two, 22 bits; K and Q are exact in fp16 (bf16
// rows scaled by a power of two), so those products take two terms and those
// with T and P T three. Sums are fp32.
//
// The chunks of one head follow on one another, X - R - U - S, and bound the
// kernel: products of 64 tokens and the conversions between them. The products
// for Y run in the gaps. Warps 0 to 3 hold the rows, warp 4 issues the products,
// warps 5 to 7 bring tiles two chunks ahead.
#include "delta_common.cuh"
#include "tensor_core.cuh"

namespace mcc1d {

namespace {

constexpr int kC = kChunk, kRowThreads = 128, kLoadThreads = 96, kThreads = kRowThreads + 32 + kLoadThreads, kStages = 2;

struct ChunkParams {
    DeltaParams d;
    const uint8_t *prepared;
    int64_t chunks;
    int32_t tiles;            // of 128 rows of V
    bool vectors_q, vectors_k, vectors_v;
};

template <int KP>
struct Stage {
    static constexpr int kPanels = KP / 64 * kPanelBytes;
    static constexpr int K = 0, Q = kPanels, kPrepared = 2 * kPanels;
    static constexpr int V = kPrepared + (kChunkBytes + 1023) / 1024 * 1024;
    static constexpr int kBytes = V + kC * kRowThreads * 2;
    static_assert(kBytes % 1024 == 0, "panels on 1024 bytes");
};

// Columns of tensor memory: sums, then operands (pairs of fp16).
enum { kX = 0, kU = 64, kQS = 128, kPR = 192, kSHi = 256, kSLo = 320, kRHi = 384, kRLo = 416, kUHi = 448, kULo = 480, kColumns = 512 };

struct Barriers {
    uint64_t full[kStages], empty[kStages], factors[kStages], x, r, u, v, y, s, end;
    uint32_t tmem;
};

// Eight 16-bit values, from `live` of them.
__device__ __forceinline__ uint4 eight(const uint16_t *from, bool vectors, int live)
{
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (vectors) {
        if (live > 0)
            r = __ldg(reinterpret_cast<const uint4 *>(from));
    } else if (live > 0) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = i < live ? __ldg(from + i) : 0u;
        r = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
    return r;
}

template <int DT>
__device__ __forceinline__ uint4 as_half(uint4 v, float scale)
{
    if constexpr (DT == 1) {
        return v;
    } else {
        const float2 s = make_float2(scale, scale);
        return make_uint4(pack_half2(mul2(unpack2<0>(v.x), s)), pack_half2(mul2(unpack2<0>(v.y), s)), pack_half2(mul2(unpack2<0>(v.z), s)),
                          pack_half2(mul2(unpack2<0>(v.w), s)));
    }
}

// Pieces of eight values of 64 rows, in the order that the loading threads
// share: all loads of a thread first, so that they are in flight together.
template <int PIECES>
struct Pieces {
    static constexpr int N = (kC * PIECES + kLoadThreads - 1) / kLoadThreads;
    uint4 v[N];
    __device__ __forceinline__ void load(const uint16_t *from, int64_t step, int width, bool vectors, int n, int thread)
    {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = thread + j * kLoadThreads, t = e / PIECES, piece = e % PIECES;
            v[j] = eight(from + t * step + 8 * piece, vectors, t < n ? width - 8 * piece : 0);
        }
    }
};

// A chunk's rows of q or k as panels.
template <int DT, int KP>
__device__ __forceinline__ void put_rows(const Pieces<KP / 8> &r, const float *scales, uint8_t *panels, int thread)
{
    constexpr int PIECES = KP / 8;
#pragma unroll
    for (int j = 0; j < Pieces<PIECES>::N; ++j) {
        const int e = thread + j * kLoadThreads, t = e / PIECES, piece = e % PIECES;
        if (t < kC)
            *reinterpret_cast<uint4 *>(panels + (piece / 8) * kPanelBytes + panel_at(t, piece % 8)) =
                as_half<DT>(r.v[j], DT == 0 ? scales[t] : 1.f);
    }
}

// Half of a thread's row of 64 values as terms: columns `hi` and `lo` on.
__device__ __forceinline__ void put_terms(const float *x, float scale, uint32_t hi, uint32_t lo)
{
    uint32_t h[16], l[16];
    const float2 s = make_float2(scale, scale);
#pragma unroll
    for (int e = 0; e < 16; ++e)
        two_terms(mul2(make_float2(x[2 * e], x[2 * e + 1]), s), h[e], l[e]);
    tmem_store(hi, h);
    tmem_store(lo, l);
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

template <int DT, int KP>
__global__ void __launch_bounds__(kThreads, 1) delta_chunks_kernel(const __grid_constant__ ChunkParams cp)
{
    typedef Stage<KP> St;
    extern __shared__ uint8_t raw_shared[];
    __shared__ Barriers bars;
    uint8_t *stages = raw_shared + (1024 - smem_u32(raw_shared) % 1024) % 1024;
    const DeltaParams &p = cp.d;
    const int tid = threadIdx.x, warp = tid / 32;
    const int item = blockIdx.x / cp.tiles, v0 = (blockIdx.x % cp.tiles) * kRowThreads;
    const int b = item / p.H, h = item % p.H, g = h / (p.H / p.G);
    const int64_t n = clamped_length(p.lengths, b, p.S), chunks = (n + kC - 1) / kC;
    const int64_t BH = (int64_t)p.B * p.H, VK = (int64_t)p.V * p.K;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&bars.full[i]), kLoadThreads);
            mbar_init(smem_u32(&bars.factors[i]), 1);
            mbar_init(smem_u32(&bars.empty[i]), kRowThreads + 1);
        }
        mbar_init(smem_u32(&bars.x), 1), mbar_init(smem_u32(&bars.u), 1), mbar_init(smem_u32(&bars.y), 1), mbar_init(smem_u32(&bars.end), 1);
        mbar_init(smem_u32(&bars.r), kRowThreads), mbar_init(smem_u32(&bars.v), kRowThreads), mbar_init(smem_u32(&bars.s), kRowThreads);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4)
        tmem_alloc(smem_u32(&bars.tmem), kColumns);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp < 4) {
        const int row = v0 + tid;
        const bool mine = row < p.V;
        const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
        float s[KP];
        {
            const float *from = p.state ? p.state + item * VK + (int64_t)row * p.K : nullptr;
#pragma unroll
            for (int k = 0; k < KP; ++k)
                s[k] = from && mine && k < p.K ? from[k] : 0.f;
        }
        float of_s = 1.f;      // what the state's terms are multiplied by
        const auto put_state = [&]() {
            const float scale = scale_for(most_of(s));
            of_s = inverse_scale(scale);
#pragma unroll
            for (int c = 0; c < KP / 32; ++c)
                put_terms(s + 32 * c, scale, lanes + kSHi + 16 * c, lanes + kSLo + 16 * c);
            tmem_wait_stores();
            tmem_fence_before();
            mbar_arrive(smem_u32(&bars.s));
        };
        const auto write_state = [&](float *to) {
            if (mine)
#pragma unroll
                for (int k = 0; k < KP; ++k)
                    if (k < p.K)
                        to[(int64_t)row * p.K + k] = s[k];
        };
        int64_t i = 0;
        if (chunks > 0)
            put_state();
        for (; i < chunks; ++i) {
            const uint32_t parity = (uint32_t)(i & 1);
            const uint8_t *stage = stages + (i % kStages) * St::kBytes;
            const float *f = reinterpret_cast<const float *>(stage + St::kPrepared + 4 * kPanelBytes);
            const uint16_t *v = reinterpret_cast<const uint16_t *>(stage + St::V) + tid;
            const int live = (int)(n - i * kC < kC ? n - i * kC : kC);
            if (p.states)
                write_state(p.states + (i * BH + item) * VK);
            // the tiles of this chunk (the products wait for them too, but this thread reads some itself)
            bool ok = mbar_wait_bounded_inline(smem_u32(&bars.full[i % kStages]), (uint32_t)(i / kStages) & 1);
            ok = ok && mbar_wait_bounded_inline(smem_u32(&bars.x), parity);
            if (!__all_sync(0xFFFFFFFFu, ok))
                break;
            tmem_fence_after();
            float r[kC], of_r;
            {
                uint32_t x[2][32];
                tmem_load(lanes + kX, x[0]);
                tmem_load(lanes + kX + 32, x[1]);
                tmem_wait(x[0]), tmem_wait(x[1]);
#pragma unroll
                for (int t = 0; t < kC; t += 4) {
                    const float4 bt = *reinterpret_cast<const float4 *>(f + kFactorB * kC + t), ft = *reinterpret_cast<const float4 *>(f + kFactorX * kC + t);
                    const float bs[4] = {bt.x, bt.y, bt.z, bt.w}, fs[4] = {ft.x, ft.y, ft.z, ft.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        r[t + e] = fmaf(-fs[e] * of_s, __uint_as_float(x[(t + e) / 32][(t + e) % 32]), bs[e] * unpack2<DT>(v[(t + e) * kRowThreads]).x);
                }
                const float scale = scale_for(most_of(r));
                of_r = inverse_scale(scale);
                put_terms(r, scale, lanes + kRHi, lanes + kRLo);
                put_terms(r + 32, scale, lanes + kRHi + 16, lanes + kRLo + 16);
                tmem_wait_stores();
                tmem_fence_before();
                mbar_arrive(smem_u32(&bars.r));
            }
            float of_u;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded_inline(smem_u32(&bars.u), parity)))
                break;
            tmem_fence_after();
            {
                uint32_t x[2][32];
                tmem_load(lanes + kU, x[0]);
                tmem_load(lanes + kU + 32, x[1]);
                tmem_wait(x[0]), tmem_wait(x[1]);
                if (p.u) {
                    float *to = p.u + (i * kC * BH + item) * p.V + row;
#pragma unroll
                    for (int t = 0; t < kC; ++t)
                        if (mine && t < live)
                            to[t * BH * p.V] = __uint_as_float(x[t / 32][t % 32]) * (of_r * f[kFactorT * kC + t]);
                }
#pragma unroll
                for (int t = 0; t < kC; t += 4) {
                    const float4 ft = *reinterpret_cast<const float4 *>(f + kFactorU * kC + t);
                    const float fs[4] = {ft.x, ft.y, ft.z, ft.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        r[t + e] = __uint_as_float(x[(t + e) / 32][(t + e) % 32]) * (fs[e] * of_r);
                }
                const float scale = scale_for(most_of(r));
                of_u = inverse_scale(scale);
                put_terms(r, scale, lanes + kUHi, lanes + kULo);
                put_terms(r + 32, scale, lanes + kUHi + 16, lanes + kULo + 16);
                tmem_wait_stores();
                tmem_fence_before();
                mbar_arrive(smem_u32(&bars.v));
            }
            const float end = f[kFactorEnd * kC];
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded_inline(smem_u32(&bars.y), parity)))
                break;
            tmem_fence_after();
            if (p.y) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t a[32], c[32];
                    tmem_load(lanes + kQS + 32 * half, a);
                    tmem_load(lanes + kPR + 32 * half, c);
                    tmem_wait(a), tmem_wait(c);
                    uint16_t *to = p.y + ((i * kC + 32 * half) * BH + item) * p.V + row;
                    const int64_t rows = p.S - (i * kC + 32 * half);
#pragma unroll
                    for (int t = 0; t < 32; ++t) {
                        const float yq = __uint_as_float(a[t]) * (of_s * f[kFactorQ * kC + 32 * half + t]);
                        const float y = fmaf(__uint_as_float(c[t]), of_r * f[kFactorP * kC + 32 * half + t], yq);
                        if (mine && t < rows)
                            to[t * BH * p.V] = t + 32 * half < live ? (uint16_t)pack2<DT>(make_float2(y, 0.f)) : (uint16_t)0;
                    }
                }
            }
            mbar_arrive(smem_u32(&bars.empty[i % kStages]));
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded_inline(smem_u32(&bars.end), parity)))
                break;
            tmem_fence_after();
#pragma unroll
            for (int c = 0; c < KP / 32; ++c) {
                uint32_t x[32];
                tmem_load(lanes + kX + 32 * c, x);
                tmem_wait(x);
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    s[32 * c + k] = fmaf(of_u, __uint_as_float(x[k]), end * s[32 * c + k]);
            }
            if (i + 1 < chunks)
                put_state();
        }
        // a wait that gave up leaves NaN behind
        const bool failed = i < chunks;
        if (failed)
#pragma unroll
            for (int k = 0; k < KP; ++k)
                s[k] = __uint_as_float(0x7FFFFFFFu);
        if (p.final_state)
            write_state(p.final_state + item * VK);
        if (p.y && mine) {
            for (int64_t t = i * kC; t < p.S; ++t)
                p.y[(t * BH + item) * p.V + row] = failed ? 0x7FFF : 0;
        }
    } else if (warp == 4) {
        if (tid % 32 == 0) {
            constexpr uint32_t rows64 = mma_kind(kC, false), columns = mma_kind(KP, true);
            for (int64_t i = 0; i < chunks; ++i) {
                const uint32_t parity = (uint32_t)(i & 1), stage = smem_u32(stages) + (uint32_t)(i % kStages) * St::kBytes;
                bool ok = mbar_wait_bounded_inline(smem_u32(&bars.full[i % kStages]), (uint32_t)(i / kStages) & 1);
                ok = ok && mbar_wait_bounded_inline(smem_u32(&bars.s), parity);
                if (!ok)
                    break;
                tmem_fence_after();
#pragma unroll
                for (int j = 0; j < KP / 16; ++j) {
                    const uint64_t k = desc_rows(stage + St::K + (j / 4) * kPanelBytes) + 2 * (j % 4);
                    mma_ts(tmem + kX, tmem + kSHi + 8 * j, k, rows64, j > 0);
                    mma_ts(tmem + kX, tmem + kSLo + 8 * j, k, rows64, true);
                }
                mma_commit(smem_u32(&bars.x));
#pragma unroll
                for (int j = 0; j < KP / 16; ++j) {
                    const uint64_t q = desc_rows(stage + St::Q + (j / 4) * kPanelBytes) + 2 * (j % 4);
                    mma_ts(tmem + kQS, tmem + kSHi + 8 * j, q, rows64, j > 0);
                    mma_ts(tmem + kQS, tmem + kSLo + 8 * j, q, rows64, true);
                }
                if (!mbar_wait_bounded_inline(smem_u32(&bars.r), parity))
                    break;
                tmem_fence_after();
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    const uint32_t d = tmem + (which ? kPR : kU), at = stage + St::kPrepared + which * 2 * kPanelBytes;
#pragma unroll
                    for (int j = 0; j < kC / 16; ++j) {
                        const uint64_t hi = desc_rows(at) + 2 * j, lo = desc_rows(at + kPanelBytes) + 2 * j;
                        mma_ts(d, tmem + kRHi + 8 * j, hi, rows64, j > 0);
                        mma_ts(d, tmem + kRHi + 8 * j, lo, rows64, true);
                        mma_ts(d, tmem + kRLo + 8 * j, hi, rows64, true);
                    }
                    mma_commit(smem_u32(which ? &bars.y : &bars.u));
                }
                if (!mbar_wait_bounded_inline(smem_u32(&bars.v), parity))
                    break;
                tmem_fence_after();
#pragma unroll
                for (int j = 0; j < kC / 16; ++j) {
                    const uint64_t k = desc_columns(stage + St::K, kPanelBytes) + (uint64_t)(2048 * j >> 4);
                    mma_ts(tmem + kX, tmem + kUHi + 8 * j, k, columns, j > 0);
                    mma_ts(tmem + kX, tmem + kULo + 8 * j, k, columns, true);
                }
                mma_commit(smem_u32(&bars.end));
                mma_commit(smem_u32(&bars.empty[i % kStages]));
            }
        }
    } else {
        const int thread = tid - kRowThreads - 32;
        for (int64_t i = 0; i < chunks; ++i) {
            const int64_t t0 = i * kC;
            const int live = (int)(n - t0 < kC ? n - t0 : kC);
            uint8_t *stage = stages + (i % kStages) * St::kBytes;
            const uint32_t full = smem_u32(&bars.full[i % kStages]), ready = smem_u32(&bars.factors[i % kStages]);
            Pieces<KP / 8> k, q;
            Pieces<kRowThreads / 8> v;
            k.load(p.k + t0 * p.k_s[0] + b * p.k_s[1] + g * p.k_s[2], p.k_s[0], p.K, cp.vectors_k, live, thread);
            q.load(p.q + t0 * p.q_s[0] + b * p.q_s[1] + g * p.q_s[2], p.q_s[0], p.K, cp.vectors_q, live, thread);
            v.load(p.v + t0 * p.v_s[0] + b * p.v_s[1] + h * p.v_s[2] + v0, p.v_s[0], p.V - v0, cp.vectors_v, live, thread);
            if (!mbar_wait_bounded_inline(smem_u32(&bars.empty[i % kStages]), (uint32_t)(i / kStages + 1) & 1))
                break;
            if (thread == 0) {
                mbar_arrive_expect_tx(ready, kChunkBytes);
                bulk_g2s(smem_u32(stage + St::kPrepared), cp.prepared + (item * cp.chunks + i) * kChunkBytes, kChunkBytes, ready);
            }
#pragma unroll
            for (int j = 0; j < Pieces<kRowThreads / 8>::N; ++j) {
                const int e = thread + j * kLoadThreads;
                if (e < kC * kRowThreads / 8)
                    *reinterpret_cast<uint4 *>(stage + St::V + 16 * e) = v.v[j];
            }
            if (!mbar_wait_bounded_inline(ready, (uint32_t)(i / kStages) & 1))
                break;
            const float *f = reinterpret_cast<const float *>(stage + St::kPrepared + 4 * kPanelBytes);
            put_rows<DT, KP>(k, f + kFactorScaleK * kC, stage + St::K, thread);
            put_rows<DT, KP>(q, f + kFactorScaleQ * kC, stage + St::Q, thread);
            shared_to_async();
            mbar_arrive(full);
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 4) {
        tmem_fence_after();
        tmem_free(tmem, kColumns);
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
    p.tiles = (int32_t)((a.V + kRowThreads - 1) / kRowThreads);
    const auto vectors = [](int64_t n, const void *at, const int64_t (&s)[3]) { return vectors_for(n, (uintptr_t)at, s[0] | s[1] | s[2]); };
    p.vectors_q = vectors(a.K, a.q, a.q_strides), p.vectors_k = vectors(a.K, a.k, a.k_strides), p.vectors_v = vectors(a.V, a.v, a.v_strides);
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
