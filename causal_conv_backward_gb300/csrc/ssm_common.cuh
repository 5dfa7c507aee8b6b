// ssm_common.cuh - device helpers of the short convolution and the selective
// scan: vectors of 16-bit channels, and the gate and softplus functions.
#pragma once

#include <type_traits>

#include "device_common.cuh"
#include "plan.h"

namespace mcc1d {

// Launches a kernel and says whether this launch failed (an error that an
// earlier call of the program left behind is not this call's).
// `after`: as a programmatic dependent of the call's kernel before it, whose
// results it waits for itself (previous_done) once it is set up.
template <class... P, class... A>
int32_t launch_as(bool after, void (*kernel)(P...), dim3 grid, int threads, int shared_bytes, cudaStream_t stream, A &&...args)
{
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = (size_t)shared_bytes;
    c.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &attr;
    c.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, P(args)...) == cudaSuccess ? kOk : kErrCuda;
}
template <class... P, class... A>
int32_t launch(void (*kernel)(P...), dim3 grid, int threads, int shared_bytes, cudaStream_t stream, A &&...args)
{
    return launch_as(false, kernel, grid, threads, shared_bytes, stream, args...);
}

// The kernel this one depends on has finished (at once where it was launched
// plainly); the kernel that depends on this one may be set up.
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

constexpr float kLog2e = 1.4426950408889634f;

// V = 8, 4, 2 or 1 adjacent 16-bit channels as P packed pairs (V = 1: one
// pair whose upper half is zero on load and dropped on store).
template <int V>
struct Vec {
    static constexpr int P = V > 1 ? V / 2 : 1;
    uint32_t u[P];
};

// Channels per thread of the short convolution over prompts: a tap costs V
// registers of weights and of each window, so wide kernels take fewer.
constexpr int conv_vec(int W) { return W <= 4 ? 4 : 2; }

// As many of them as the addresses (their bits or'd) and the row steps in
// elements (or'd) allow: 4, 2 or 1.
inline int conv_vec_for(int W, uintptr_t addresses, int64_t steps)
{
    int V = conv_vec(W);
    while (V > 1 && ((addresses & (uintptr_t)(2 * V - 1)) != 0 || (steps & (V - 1)) != 0))
        V /= 2;
    return V;
}

template <int V>
__device__ __forceinline__ Vec<V> vzero()
{
    Vec<V> r;
#pragma unroll
    for (int i = 0; i < Vec<V>::P; ++i)
        r.u[i] = 0u;
    return r;
}

template <int V>
__device__ __forceinline__ Vec<V> vload(const uint16_t *p)
{
    Vec<V> r;
    if constexpr (V == 8) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        r.u[0] = v.x;
        r.u[1] = v.y;
        r.u[2] = v.z;
        r.u[3] = v.w;
    } else if constexpr (V == 4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        r.u[0] = v.x;
        r.u[1] = v.y;
    } else if constexpr (V == 2) {
        r.u[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    } else {
        r.u[0] = __ldg(p);
    }
    return r;
}

template <int V>
__device__ __forceinline__ void vstore(uint16_t *p, const Vec<V> &r)
{
    if constexpr (V == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(r.u[0], r.u[1], r.u[2], r.u[3]);
    else if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(p) = make_uint2(r.u[0], r.u[1]);
    else if constexpr (V == 2)
        *reinterpret_cast<uint32_t *>(p) = r.u[0];
    else
        *p = (uint16_t)r.u[0];
}

// Asynchronous copy of V channels (4 or 8 bytes) from global to shared memory,
// in the issuing thread's groups.
template <int V>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint16_t *src)
{
    static_assert(V == 2 || V == 4, "4 or 8 bytes");
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(2 * V) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the N newest groups of this thread have arrived.
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int V>
__device__ __forceinline__ Vec<V> vload_shared(const uint8_t *p)
{
    Vec<V> r;
    if constexpr (V == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.u[0] = v.x;
        r.u[1] = v.y;
    } else {
        r.u[0] = *reinterpret_cast<const uint32_t *>(p);
    }
    return r;
}

// Rows of T tensors on their way to one thread: whole batches of R rows, STAGES
// of them, copied asynchronously into shared memory, where the thread reads
// back only what it copied itself (no barrier). Registers could not hold the
// bytes that have to be in flight: at about 0.8 us of latency an SM needs
// 36 KB. Single channels (V = 1) are too narrow to copy and wait in registers.
template <int V, int T, int R, int STAGES>
struct RowRing {
    static constexpr int BYTES_PER_THREAD = V == 1 ? 0 : T * R * STAGES * 2 * V;
    const uint16_t *src[T];
    int64_t step[T];
    int64_t left;          // rows not yet asked for
    uint8_t *slots;        // of the block: slot (stage, row, tensor) of thread i at ((stage R + row) T + tensor) threads + i
    int threads, next_in, next_out;
    Vec<V> hold[V == 1 ? T * R : 1];

    __device__ __forceinline__ uint8_t *slot(int stage, int row, int tensor) const
    {
        return slots + (((stage * R + row) * T + tensor) * threads + threadIdx.x) * (2 * V);
    }
    __device__ __forceinline__ void ask()
    {
        if constexpr (V > 1) {
            if (left >= R) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int t = 0; t < T; ++t) {
                        copy_async<V>(smem_u32(slot(next_in, r, t)), src[t]);
                        src[t] += step[t];
                    }
                left -= R;
            }
            copy_commit();
            next_in = next_in + 1 == STAGES ? 0 : next_in + 1;
        } else if (left >= R) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    hold[r * T + t] = vload<V>(src[t]);
                    src[t] += step[t];
                }
            left -= R;
        }
    }
    __device__ __forceinline__ void start()
    {
        next_in = next_out = 0;
#pragma unroll
        for (int s = 0; s < (V > 1 ? STAGES - 1 : 1); ++s)
            ask();
    }
    // The next batch; the one STAGES - 1 after it is asked for.
    __device__ __forceinline__ void take(Vec<V> (&out)[R * T])
    {
        if constexpr (V > 1) {
            ask();
            copy_wait<STAGES - 1>();
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int t = 0; t < T; ++t)
                    out[r * T + t] = vload_shared<V>(slot(next_out, r, t));
            next_out = next_out + 1 == STAGES ? 0 : next_out + 1;
        } else {
#pragma unroll
            for (int i = 0; i < R * T; ++i)
                out[i] = hold[i];
            ask();
        }
    }
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// exp(dt A) for two states, from A log2 e. ex2.approx comes out low by 0.6 to
// 2.6e-8 of its result on average for exponents between -1 and 0 (measured
// over 2^20 points a decade; 2^0 is exact), and a decay close to 1 is applied
// thousands of times before a state is forgotten, so the bias adds up where
// rounding would cancel. kDecayShift in the exponent, free in the multiply-add,
// takes the middle of it out: grad A's error on 16 K tokens and 16384 channels
// of slow decays fell from 1.74e-6 to 0.78e-6. ex2(kDecayShift) is still 1.
constexpr float kDecayShift = 2.0e-8f;
__device__ __forceinline__ float2 decay2(float2 dt2, float2 A2)
{
    const float2 x = fma2(dt2, A2, make_float2(kDecayShift, kDecayShift));
    return make_float2(ex2(x.x), ex2(x.y));
}

// exp(dt A) h + b for two states, from A log2 e and the dt of many tokens. The
// growth goes in as two factors, neither of them infinite: alone it may pass
// fp32 where no state does (an h of zero stays zero); token by token it does
// not arise.
__device__ __forceinline__ float2 grown(float2 h, float dt, float2 A2, float2 b)
{
    const float2 x = mul2(make_float2(0.5f * dt, 0.5f * dt), A2);
    const float2 f = make_float2(ex2(fminf(x.x, 127.f)), ex2(fminf(x.y, 127.f)));
    return fma2(f, mul2(f, h), b);
}

__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-x): e^-x overflows to infinity below -88, where the reciprocal is 0.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.0f + ex2(-kLog2e * x)); }

__device__ __forceinline__ float2 sigmoid2(float2 x)
{
    const float2 t = mul2(x, make_float2(-kLog2e, -kLog2e));
    const float2 d = add2(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
    return make_float2(rcp(d.x), rcp(d.y));
}

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x|, and log(1 + e) = 2 atanh(s)
// with s = e / (2 + e) <= 1/3: an odd series in s, so the result keeps its
// relative accuracy where e, and with it the step, is small (log2 of 1 + e
// would not). The polynomial in s^2 is a least-squares fit, weighted to equal
// ripple, of atanh(s)/s on [0, 1/9]: off by 8e-9 of it. -|x| log2 e is carried in two parts, since its
// rounding alone would cost |x| 2^-24.
__device__ __forceinline__ float2 softplus2(float2 x)
{
    // held above -100, where e is 0: an infinite x leaves no infinity minus infinity in lo
    const float2 m = make_float2(-fminf(fabsf(x.x), 100.f), -fminf(fabsf(x.y), 100.f));
    const float2 L = make_float2(kLog2e, kLog2e);
    const float2 t = mul2(m, L);
    float2 lo = fma2(m, L, make_float2(-t.x, -t.y));
    lo = fma2(m, make_float2(1.925963e-8f, 1.925963e-8f), lo);   // log2 e - kLog2e
    float2 e = make_float2(ex2(t.x), ex2(t.y));
    e = fma2(mul2(lo, make_float2(0.6931472f, 0.6931472f)), e, e);
    const float2 d = add2(e, make_float2(2.f, 2.f));
    const float2 s = mul2(e, make_float2(rcp(d.x), rcp(d.y)));
    const float2 q = mul2(s, s);
    float2 r = fma2(q, make_float2(0.140891641f, 0.140891641f), make_float2(0.139803022f, 0.139803022f));
    r = fma2(r, q, make_float2(0.200124547f, 0.200124547f));
    r = fma2(r, q, make_float2(0.333331585f, 0.333331585f));
    r = fma2(r, q, make_float2(1.f, 1.f));
    return fma2(add2(s, s), r, make_float2(x.x < 0.f ? 0.f : x.x, x.y < 0.f ? 0.f : x.y));   // NaN stays NaN
}

__device__ __forceinline__ float softplus(float x) { return softplus2(make_float2(x, x)).x; }

// A sequence's length, held to 0..S.
__device__ __forceinline__ int64_t clamped_length(const int32_t *lengths, int64_t b, int64_t S)
{
    if (!lengths)
        return S;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n > S ? S : n);
}

}  // namespace mcc1d
