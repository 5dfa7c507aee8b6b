// norm_common.cuh - rows of values spread over threads: addresses, loads,
// sums, and the choice of threads per row.
//
// All four kernels move each input and output once and do some ten operations
// a value, so HBM bounds them: a row stays in registers from its load to its
// store, and threads hold 16-byte vectors, E values each.
#pragma once

#include "norm.h"
#include "ssm_common.cuh"

namespace mcc1d {

// r / d and r % d for r < 2^31 by one multiplication: with l = ceil(log2 d) and
// m = floor(2^(31+l) / d) + 1, floor(r m / 2^(31+l)) is the quotient (the excess
// r (m d - 2^(31+l)) / (d 2^(31+l)) is at most r / 2^(31+l) <= 1/d' for d' >= d).
struct Divisor {
    uint32_t d;
    uint32_t shift;
    uint64_t m;
    Divisor() = default;
    explicit Divisor(int64_t by) : d((uint32_t)by)
    {
        uint32_t l = 0;
        while (((uint64_t)1 << l) < d)
            ++l;
        shift = 31 + l;
        m = ((uint64_t)1 << shift) / d + 1;
    }
    __device__ __forceinline__ uint32_t quotient(uint32_t r) const { return (uint32_t)((r * m) >> shift); }
};

// The address of row r = (s B + b) H + h of a tensor with these strides.
struct RowAddress {
    int64_t s, b, h;
};
struct RowOrder {
    Divisor B, H;
    __device__ __forceinline__ int64_t at(const RowAddress &a, uint32_t r) const
    {
        const uint32_t q = H.quotient(r), s = B.quotient(q);
        return s * a.s + (q - s * B.d) * a.b + (r - q * H.d) * a.h;
    }
};

// A row of up to V x NV x TPR values over TPR threads: vector j of thread t
// starts at value (j TPR + t) V.
template <int V_, int NV_, int TPR_>
struct RowShape {
    static constexpr int V = V_, NV = NV_, TPR = TPR_, E = V_ * NV_;
    static constexpr int THREADS = TPR_ > 32 ? TPR_ : 256, ROWS = THREADS / TPR_;
};

template <class R>
__device__ __forceinline__ int thread_of_row() { return threadIdx.x % R::TPR; }

// Two neighbours of a thread's values, for packed arithmetic.
template <int N>
__device__ __forceinline__ float2 pair(const float (&x)[N], int e) { return make_float2(x[e], x[e + 1]); }
template <int N>
__device__ __forceinline__ void put(float (&x)[N], int e, float2 v) { x[e] = v.x, x[e + 1] = v.y; }

// ------------------------------------------------------------------ loads and stores
// 16-bit values of type DT (0, 1), or fp32 (2); zero past the row's end.
template <int DT>
struct Element {
    typedef uint16_t type;
};
template <>
struct Element<2> {
    typedef float type;
};

// One thread's share of a row as it came from memory.
template <int DT, class R>
struct Share {
    static constexpr int WORDS = R::V == 1 ? 1 : (DT == 2 ? 8 : 4);
    uint32_t u[R::NV * WORDS];
};

template <int DT, class R>
__device__ __forceinline__ Share<DT, R> load_share(const void *base, int64_t at, int D)
{
    Share<DT, R> r;
    const typename Element<DT>::type *p = static_cast<const typename Element<DT>::type *>(base) + at;
    constexpr int W = Share<DT, R>::WORDS;
#pragma unroll
    for (int j = 0; j < R::NV; ++j) {
        const int i = (j * R::TPR + thread_of_row<R>()) * R::V;
#pragma unroll
        for (int w = 0; w < W; ++w)
            r.u[j * W + w] = 0u;
        if (i < D) {
            if constexpr (R::V == 1 && DT == 2) {
                r.u[j] = __float_as_uint(__ldg(p + i));
            } else if constexpr (R::V == 1) {
                r.u[j] = __ldg(p + i);
            } else {
#pragma unroll
                for (int w = 0; w < W; w += 4) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p + i) + w / 4);
                    r.u[j * W + w] = v.x, r.u[j * W + w + 1] = v.y, r.u[j * W + w + 2] = v.z, r.u[j * W + w + 3] = v.w;
                }
            }
        }
    }
    return r;
}

template <int DT, class R>
__device__ __forceinline__ void values(const Share<DT, R> &r, float (&x)[R::E])
{
    constexpr int W = Share<DT, R>::WORDS;
#pragma unroll
    for (int j = 0; j < R::NV; ++j) {
        if constexpr (DT == 2) {
#pragma unroll
            for (int e = 0; e < R::V; ++e)
                x[j * R::V + e] = __uint_as_float(r.u[j * W + e]);
        } else if constexpr (R::V == 1) {
            x[j] = unpack2<DT>(r.u[j]).x;
        } else {
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float2 v = unpack2<DT>(r.u[j * W + w]);
                x[j * R::V + 2 * w] = v.x, x[j * R::V + 2 * w + 1] = v.y;
            }
        }
    }
}

template <int DT, class R>
__device__ __forceinline__ void load_values(const void *base, int64_t at, int D, float (&x)[R::E])
{
    values<DT, R>(load_share<DT, R>(base, at, D), x);
}

template <int DT, class R>
__device__ __forceinline__ void store_values(void *base, int64_t at, int D, const float (&x)[R::E])
{
    typename Element<DT>::type *p = static_cast<typename Element<DT>::type *>(base) + at;
#pragma unroll
    for (int j = 0; j < R::NV; ++j) {
        const int i = (j * R::TPR + thread_of_row<R>()) * R::V;
        if (i >= D)
            continue;
        const float *v = x + j * R::V;
        if constexpr (R::V == 1 && DT == 2) {
            p[i] = v[0];
        } else if constexpr (R::V == 1) {
            p[i] = (uint16_t)pack2<DT>(make_float2(v[0], 0.f));
        } else if constexpr (DT == 2) {
            float4 *q = reinterpret_cast<float4 *>(p + i);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(p + i) = make_uint4(pack2<DT>(make_float2(v[0], v[1])), pack2<DT>(make_float2(v[2], v[3])),
                                                           pack2<DT>(make_float2(v[4], v[5])), pack2<DT>(make_float2(v[6], v[7])));
        }
    }
}

// ------------------------------------------------------------------ sums over a row
// N sums over the threads of a row, the same for each of them. `turn` flips
// between calls, so that one barrier a call is enough.
template <class R, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*shared)[2][3][32], int &turn)
{
#pragma unroll
    for (int d = (R::TPR < 32 ? R::TPR : 32) / 2; d > 0; d /= 2)
#pragma unroll
        for (int k = 0; k < N; ++k)
            v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], d);
    if constexpr (R::TPR > 32) {
        constexpr int WARPS = R::TPR / 32;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int k = 0; k < N; ++k)
                (*shared)[turn][k][threadIdx.x / 32] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                s += (*shared)[turn][k][w];
            v[k] = s;
        }
        turn ^= 1;
    }
}

// 1 / sqrt(v), to the last bits: the instruction's result and one Newton step
// (not at 0 and infinity, where the step would make NaN of them).
__device__ __forceinline__ float inverse_root(float v)
{
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    if (r > 0.f && r < INFINITY)
        r = r * fmaf(-0.5f * v * r, r, 1.5f);
    return r;
}

// ------------------------------------------------------------------ which threads
// Threads for rows of D values: up to 1024 a warp or less, so that sums need
// shuffles only; above, a block. A thread's values past the row's end cost as much
// as the others: 2^27 values in rows of 128, 256, 1024, 2048 and 4096 take 117 to 136
// us in the gated norm in shapes of their width, and 212 to 370 in the next wider one.
// So there is a shape for every power of two, and two between (up to 1536 and 2560),
// and other widths have up to half of a shape idle. Rows of 513 to 1024 values with an
// fp32 residual do not fit the residual norm's registers whole (0.7 KB a thread
// spilled), nor do rows above 8192 in the gradients (0.4 KB). Rows that cannot be read
// in 16-byte vectors are read value by value, 172 to 317 us at these widths.
template <class F>
int32_t with_row_shape(int64_t D, bool vectors, F &&f)
{
    if (vectors) {
        if (D <= 64)
            return f(RowShape<8, 1, 8>());
        if (D <= 128)
            return f(RowShape<8, 1, 16>());
        if (D <= 256)
            return f(RowShape<8, 1, 32>());
        if (D <= 512)
            return f(RowShape<8, 2, 32>());
        if (D <= 1024)
            return f(RowShape<8, 4, 32>());
        if (D <= 1536)
            return f(RowShape<8, 2, 96>());
        if (D <= 2048)
            return f(RowShape<8, 2, 128>());
        if (D <= 2560)
            return f(RowShape<8, 2, 160>());
        if (D <= 4096)
            return f(RowShape<8, 2, 256>());
        if (D <= 8192)
            return f(RowShape<8, 2, 512>());
        return f(RowShape<8, 2, 1024>());
    }
    if (D <= 64)
        return f(RowShape<1, 2, 32>());
    if (D <= 128)
        return f(RowShape<1, 4, 32>());
    if (D <= 256)
        return f(RowShape<1, 8, 32>());
    if (D <= 512)
        return f(RowShape<1, 16, 32>());
    if (D <= 1024)
        return f(RowShape<1, 16, 64>());
    if (D <= 2048)
        return f(RowShape<1, 16, 128>());
    if (D <= 4096)
        return f(RowShape<1, 16, 256>());
    if (D <= 8192)
        return f(RowShape<1, 16, 512>());
    return f(RowShape<1, 16, 1024>());
}

// The backwards hold sums and the next row too: half as many values to a thread
// (rows of 2048 of the residual norm, 193 us with sixteen to a thread, 147 with
// eight), up to 4096. Above, sixteen with the sums in shared memory: 2^27 values in
// rows of 8192 take 302 us in the gated and 403 in the residual norm's gradients,
// 1054 and 976 with sums and next row in registers, which overflow.
template <class F>
int32_t with_row_shape_bwd(int64_t D, bool vectors, F &&f)
{
    if (vectors) {
        if (D <= 64)
            return f(RowShape<8, 1, 8>());
        if (D <= 128)
            return f(RowShape<8, 1, 16>());
        if (D <= 256)
            return f(RowShape<8, 1, 32>());
        if (D <= 512)
            return f(RowShape<8, 1, 64>());
        if (D <= 1024)
            return f(RowShape<8, 1, 128>());
        if (D <= 1536)
            return f(RowShape<8, 1, 192>());
        if (D <= 2048)
            return f(RowShape<8, 1, 256>());
        if (D <= 4096)
            return f(RowShape<8, 1, 512>());
        if (D <= 8192)
            return f(RowShape<8, 2, 512>());
        return f(RowShape<8, 2, 1024>());
    }
    if (D <= 64)
        return f(RowShape<1, 2, 32>());
    if (D <= 128)
        return f(RowShape<1, 4, 32>());
    if (D <= 256)
        return f(RowShape<1, 8, 32>());
    if (D <= 512)
        return f(RowShape<1, 8, 64>());
    if (D <= 1024)
        return f(RowShape<1, 8, 128>());
    if (D <= 2048)
        return f(RowShape<1, 8, 256>());
    if (D <= 4096)
        return f(RowShape<1, 8, 512>());
    if (D <= 8192)
        return f(RowShape<1, 16, 512>());
    return f(RowShape<1, 16, 1024>());
}

// Whether rows of D values can be read in vectors of eight: addresses (or'd) on
// 16 bytes, steps in elements (or'd) and the row itself multiples of eight.
inline bool vectors_for(int64_t D, uintptr_t addresses, int64_t steps)
{
    return D % 8 == 0 && (addresses & 15u) == 0 && (steps & 7) == 0;
}

// ------------------------------------------------------------------ sums over rows
// N sums of each of a thread's values over its rows: in registers, or, where the
// rows are so long that these are needed for a row, in shared memory. Then the
// next row is not asked for ahead either.
template <class R, int N>
struct Totals {
    static constexpr bool HELD = R::E <= 8;
    static constexpr int BYTES = HELD ? 0 : N * R::E * R::TPR * 4;
    float held[N][HELD ? R::E : 2];
    float2 *at;

    __device__ __forceinline__ explicit Totals(uint8_t *shared) : at(reinterpret_cast<float2 *>(shared) + thread_of_row<R>())
    {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int e = 0; e < R::E; e += 2)
                if constexpr (HELD)
                    put(held[k], e, make_float2(0.f, 0.f));
                else
                    at[(k * R::E + e) / 2 * R::TPR] = make_float2(0.f, 0.f);
    }
    __device__ __forceinline__ void add(int k, int e, float2 a, float2 b)
    {
        if constexpr (HELD) {
            put(held[k], e, fma2(a, b, pair(held[k], e)));
        } else {
            float2 &x = at[(k * R::E + e) / 2 * R::TPR];
            x = fma2(a, b, x);
        }
    }
    __device__ __forceinline__ void get(int k, float (&x)[R::E]) const
    {
#pragma unroll
        for (int e = 0; e < R::E; e += 2)
            if constexpr (HELD)
                put(x, e, pair(held[k], e));
            else
                put(x, e, at[(k * R::E + e) / 2 * R::TPR]);
    }
};
template <class R, int N, class K, class P>
int32_t launch_totals(K kernel, int64_t blocks, cudaStream_t stream, const P &p)
{
    constexpr int bytes = Totals<R, N>::BYTES;
    if (bytes > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return kErrCuda;
    return launch(kernel, dim3((unsigned)blocks), R::THREADS, bytes, stream, p);
}

// Each thread's sums over its rows, joined over the block's rows of threads and
// written to part [blocks][D]: one barrier per use of `shared`.
template <class R>
__device__ __forceinline__ void store_part(const float (&x)[R::E], float *part, int D, float (*shared)[R::ROWS > 1 ? R::ROWS * R::TPR * R::E : 1])
{
    float sum[R::E];
#pragma unroll
    for (int e = 0; e < R::E; ++e)
        sum[e] = x[e];
    if constexpr (R::ROWS > 1) {
        __syncthreads();
        const int row = threadIdx.x / R::TPR, t = thread_of_row<R>();
#pragma unroll
        for (int e = 0; e < R::E; ++e)
            (*shared)[(row * R::E + e) * R::TPR + t] = x[e];
        __syncthreads();
        if (row > 0)
            return;
        for (int k = 1; k < R::ROWS; ++k)
#pragma unroll
            for (int e = 0; e < R::E; ++e)
                sum[e] += (*shared)[(k * R::E + e) * R::TPR + t];
    }
    float *to = part + (int64_t)blockIdx.x * D;
#pragma unroll
    for (int j = 0; j < R::NV; ++j)
#pragma unroll
        for (int e = 0; e < R::V; ++e) {
            const int i = (j * R::TPR + thread_of_row<R>()) * R::V + e;
            if (i < D)
                to[i] = sum[j * R::V + e];
        }
}

}  // namespace mcc1d
