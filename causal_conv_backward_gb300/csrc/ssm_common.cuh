// ssm_common.cuh - device helpers of the short convolution and the selective
// scan: vectors of 16-bit channels, and the gate and softplus functions.
#pragma once

#include <type_traits>

#include "device_common.cuh"

namespace mcc1d {

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

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / (1 + e^-x): e^-x overflows to infinity below -88, where the quotient is 0.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + ex2(-kLog2e * x)); }

// A sequence's length, held to 0..S.
__device__ __forceinline__ int64_t clamped_length(const int32_t *lengths, int64_t b, int64_t S)
{
    if (!lengths)
        return S;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : (n > S ? S : n);
}

}  // namespace mcc1d
