// delta_join.cu - states passed on from segment to segment of the time axis.
//
// Rows of a state are independent: a block takes eight rows of one head through
// all segments, reading each segment's K x K matrix from shared memory while the
// next one's is on its way. 25 segments of 6 heads of 64 x 64 take 40 us.
#include "delta_common.cuh"

namespace mcc1d {

namespace {

constexpr int kRows = 8, kThreads = 256;

struct JoinParams {
    float *states;
    const float *turns;
    int64_t heads;
    int32_t V, K, tiles, segments;
};

// A matrix [K,K], words in flight; rows KP + 4 apart, so that neither rows nor
// columns of it meet on a bank. Words past K are zeros.
template <int KP>
__device__ __forceinline__ void bring(float (*to)[KP + 4], const float *from, int K)
{
    for (int e = threadIdx.x; e < KP * KP; e += kThreads) {
        const int j = e / KP, k = e % KP;
        const bool there = j < K && k < K;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(&to[j][k])), "l"(from + (there ? (int64_t)j * K + k : 0)), "r"(there ? 4 : 0)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int KP, bool BACK>
__global__ void __launch_bounds__(kThreads, 1) mcc1d_delta_join_segments(const __grid_constant__ JoinParams p)
{
    extern __shared__ __align__(16) float shared[];
    typedef float Matrix[KP + 4];
    Matrix *turn[2] = {reinterpret_cast<Matrix *>(shared), reinterpret_cast<Matrix *>(shared) + KP};
    __shared__ __align__(16) float s[kRows][KP];
    constexpr int PER = kRows * KP / kThreads;       // values of a thread: one key, rows kThreads / KP apart
    const int k = threadIdx.x % KP, r0 = threadIdx.x / KP;
    const int64_t item = blockIdx.x / p.tiles, VK = (int64_t)p.V * p.K, KK = (int64_t)p.K * p.K;
    const int v0 = (blockIdx.x % p.tiles) * kRows, joins = p.segments - 2;
    // the state that leaves the first segment (of the direction) is there
    const auto at = [&](int j) { return (int64_t)(BACK ? p.segments - 2 - j : j) * p.heads + item; };
    const auto turn_at = [&](int j) { return (int64_t)(BACK ? p.segments - 1 - j : j) * p.heads + item; };
    float *state = p.states + at(0) * VK;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
        const int r = r0 + e * (kThreads / KP);
        s[r][k] = v0 + r < p.V && k < p.K ? state[(int64_t)(v0 + r) * p.K + k] : 0.f;
    }
    if (joins > 0)
        bring<KP>(turn[1], p.turns + turn_at(1) * KK, p.K);
    for (int j = 1; j <= joins; ++j) {
        if (j < joins) {
            bring<KP>(turn[(j + 1) & 1], p.turns + turn_at(j + 1) * KK, p.K);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const Matrix *m = turn[j & 1];
        state = p.states + at(j) * VK;
        float x[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int r = r0 + e * (kThreads / KP);
            x[e] = v0 + r < p.V && k < p.K ? state[(int64_t)(v0 + r) * p.K + k] : 0.f;
        }
#pragma unroll 4
        for (int i = 0; i < KP; i += 4) {
            float w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                w[c] = BACK ? m[k][i + c] : m[i + c][k];
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const float4 v = *reinterpret_cast<const float4 *>(&s[r0 + e * (kThreads / KP)][i]);
                x[e] = fmaf(v.x, w[0], fmaf(v.y, w[1], fmaf(v.z, w[2], fmaf(v.w, w[3], x[e]))));
            }
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int r = r0 + e * (kThreads / KP);
            s[r][k] = x[e];
            if (v0 + r < p.V && k < p.K)
                state[(int64_t)(v0 + r) * p.K + k] = x[e];
        }
    }
}

template <int KP, bool BACK>
int32_t join(const JoinParams &p, cudaStream_t stream)
{
    constexpr int bytes = 2 * KP * (KP + 4) * 4;
    if (cudaFuncSetAttribute(mcc1d_delta_join_segments<KP, BACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return kErrCuda;
    return launch(mcc1d_delta_join_segments<KP, BACK>, dim3((unsigned)(p.heads * p.tiles)), kThreads, bytes, stream, p);
}

}  // namespace

int32_t launch_delta_join(float *states, const float *turns, int64_t heads, int32_t V, int32_t K, int32_t segments, bool back, cudaStream_t stream)
{
    const JoinParams p = {states, turns, heads, V, K, (V + kRows - 1) / kRows, segments};
    if (back)
        return K <= 64 ? join<64, true>(p, stream) : join<128, true>(p, stream);
    return K <= 64 ? join<64, false>(p, stream) : join<128, false>(p, stream);
}

}  // namespace mcc1d
