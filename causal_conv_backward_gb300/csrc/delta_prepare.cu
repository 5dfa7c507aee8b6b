// delta_prepare.cu - a chunk's products of tokens with tokens.
//
// With c(t) the running sum of log a, D(t,i) = exp(c(t) - c(i)):
//   L(t,i) = b(t) D (k'(t).k'(i)), i < t;   P(t,i) = D (q'(t).k'(i)), i <= t
//   T = (I + L)^-1,   so that U = T R for R = b (V - e^c K' S^T),  and P U = (P T) R
// T and P T leave as two fp16 terms each (22 bits), rows scaled by powers of two,
// in the layout that delta_chunks.cu multiplies from.
//
// k'.k' and q'.k' are taken of the 16-bit tensors themselves on the tensor cores
// (their products are exact in fp32) and scaled afterwards. The inverse is that
// of the 16-wide diagonal blocks by substitution, joined twice:
// [[A,0],[C,B]]^-1 = [[A',0],[-B' C A',B']].
#include "delta_common.cuh"
#include "tensor_core.cuh"

namespace mcc1d {

namespace {

constexpr int kC = kChunk, kThreads = 256, kRow = kC + 4;

struct PrepareParams {
    DeltaParams d;
    uint8_t *out;
    int64_t chunks;
};

template <int KP>
struct PrepareShared {
    static constexpr int RS = KP + 8;                       // of 16-bit rows, so that eight of them start on different banks
    uint16_t q[kC][RS], k[kC][RS];
    float kk[kC][kRow], qk[kC][kRow];
    float L[kC][kRow], T[kC][kRow], P[kC][kRow], X[kC][kRow];
    float ch[kC], cl[kC], b[kC], fq[kC], fk[kC], lk[kC], mq[kC], mk[kC], of_v[kC], of_s[kC], of_r[kC];
};

template <int DT>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    if constexpr (DT == 0)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// out (16 rows from r0, columns from c0, `NB` of eight) = rows x columns products over KP values.
template <int DT, int KP, int NB>
__device__ __forceinline__ void token_products(const uint16_t (*rows)[KP + 8], const uint16_t (*cols)[KP + 8], const float *fr, const float *fc,
                                               float scale, float (*out)[kRow], int r0, int c0)
{
    const int lane = threadIdx.x % 32, g = lane / 4, p = 2 * (lane % 4);
    float acc[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
        acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
    for (int at = 0; at < KP; at += 16) {
        const uint32_t a[4] = {*reinterpret_cast<const uint32_t *>(&rows[r0 + g][at + p]), *reinterpret_cast<const uint32_t *>(&rows[r0 + g + 8][at + p]),
                               *reinterpret_cast<const uint32_t *>(&rows[r0 + g][at + p + 8]),
                               *reinterpret_cast<const uint32_t *>(&rows[r0 + g + 8][at + p + 8])};
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const uint32_t b[2] = {*reinterpret_cast<const uint32_t *>(&cols[c0 + 8 * n + g][at + p]),
                                   *reinterpret_cast<const uint32_t *>(&cols[c0 + 8 * n + g][at + p + 8])};
            mma16816<DT>(acc[n], a, b);
        }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = r0 + g + 8 * (e / 2), c = c0 + 8 * n + p + e % 2;
            out[r][c] = acc[n][e] * (fr[r] * scale) * fc[c];
        }
}

// to[r0+i][c0+j] = sign * sum over m < N of a[ar+i][ac+m] b[br+m][bc+j], N x N, by `threads` threads.
template <int N>
__device__ __forceinline__ void small_product(float (*to)[kRow], int r0, int c0, const float (*a)[kRow], int ar, int ac, const float (*b)[kRow],
                                              int br, int bc, float sign, int thread, int threads)
{
    for (int e = thread; e < N * N / 4; e += threads) {
        const int i = e / (N / 4), j = 4 * (e % (N / 4));
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int m = 0; m < N; ++m) {
            const float x = a[ar + i][ac + m];
            const float4 y = *reinterpret_cast<const float4 *>(&b[br + m][bc + j]);
            s.x = fmaf(x, y.x, s.x), s.y = fmaf(x, y.y, s.y), s.z = fmaf(x, y.z, s.z), s.w = fmaf(x, y.w, s.w);
        }
        *reinterpret_cast<float4 *>(&to[r0 + i][c0 + j]) = make_float4(sign * s.x, sign * s.y, sign * s.z, sign * s.w);
    }
}

// Row t of a matrix as two panels, scaled; four threads to a row, 16 values each.
// Returns 1 / scale and the sum of the row's magnitudes.
__device__ __forceinline__ float2 store_terms(const float *row, uint8_t *hi, uint8_t *lo, int t, int part)
{
    float x[16], most = 0.f, sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(row + 16 * part + j);
        x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
        most = fmaxf(most, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
        sum += (fabsf(v.x) + fabsf(v.y)) + (fabsf(v.z) + fabsf(v.w));
    }
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    }
    const float scale = scale_for(most);
#pragma unroll
    for (int piece = 0; piece < 2; ++piece) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            two_terms(make_float2(x[8 * piece + 2 * e] * scale, x[8 * piece + 2 * e + 1] * scale), h[e], l[e]);
        const uint32_t at = panel_at(t, 2 * part + piece);
        *reinterpret_cast<uint4 *>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
    return make_float2(inverse_scale(scale), sum);
}

template <int DT, int KP>
__global__ void __launch_bounds__(kThreads, 2) delta_prepare_kernel(const __grid_constant__ PrepareParams pp)
{
    extern __shared__ __align__(16) uint8_t raw_shared[];
    PrepareShared<KP> &sh = *reinterpret_cast<PrepareShared<KP> *>(raw_shared);
    const DeltaParams &p = pp.d;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int g = blockIdx.x % p.G, b = (blockIdx.x / p.G) % p.B, per = p.H / p.G;
    const int64_t chunk = blockIdx.x / p.G / p.B, t0 = chunk * kC;
    const int64_t length = clamped_length(p.lengths, b, p.S);
    if (length <= t0)
        return;
    const int n = (int)(length - t0 < kC ? length - t0 : kC);

    // q, k, their factors, and the scale that makes rows of about one size of them in fp16, without loss
    for (int i = warp; i < kC; i += kThreads / 32) {
        const uint16_t *qp = p.q + (t0 + i) * p.q_s[0] + b * p.q_s[1] + g * p.q_s[2];
        const uint16_t *kp = p.k + (t0 + i) * p.k_s[0] + b * p.k_s[1] + g * p.k_s[2];
        float sums[2] = {0.f, 0.f}, most[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KP / 32; ++j) {
            const int at = j * 32 + lane;
            const uint16_t q = i < n && at < p.K ? __ldg(qp + at) : 0, k = i < n && at < p.K ? __ldg(kp + at) : 0;
            sh.q[i][at] = q, sh.k[i][at] = k;
            const float qv = unpack2<DT>(q).x, kv = unpack2<DT>(k).x;
            sums[0] = fmaf(qv, qv, sums[0]), sums[1] = fmaf(kv, kv, sums[1]);
            most[0] = fmaxf(most[0], fabsf(qv)), most[1] = fmaxf(most[1], fabsf(kv));
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sums[e] += __shfl_xor_sync(0xFFFFFFFFu, sums[e], d);
                most[e] = fmaxf(most[e], __shfl_xor_sync(0xFFFFFFFFu, most[e], d));
            }
        if (lane == 0) {
            sh.fq[i] = unit_factor(p.flags, sums[0]), sh.fk[i] = unit_factor(p.flags, sums[1]);
            sh.lk[i] = sqrtf(sums[1]) * sh.fk[i];
            sh.mq[i] = scale_for(most[0]), sh.mk[i] = scale_for(most[1]);
        }
    }
    __syncthreads();
    // eight warps: 16 rows of one product and half of its columns each, two products
    token_products<DT, KP, 4>(sh.k, sh.k, sh.fk, sh.fk, 1.f, sh.kk, 16 * (warp % 4), 32 * (warp / 4));
    token_products<DT, KP, 4>(sh.q, sh.k, sh.fq, sh.fk, p.scale, sh.qk, 16 * (warp % 4), 32 * (warp / 4));

    for (int h = g * per; h < (g + 1) * per; ++h) {
        const int64_t item = (int64_t)b * p.H + h;
        uint8_t *out = pp.out + (item * pp.chunks + chunk) * kChunkBytes;
        float *factors = reinterpret_cast<float *>(out + 4 * kPanelBytes);
        __syncthreads();
        // gates, and the running sum of log2 a in two parts whose differences are
        // exact in the first: multiples of 2^-9 below 2^14
        if (tid < kC) {
            const int64_t t = t0 + tid;
            Gates gate = {0.f, 0.f, 0.f, 0.f};
            if (tid < n)
                gate = gates_of(p.flags, p.delta != nullptr, p.delta ? value<DT>(p.delta + t * p.delta_s[0] + b * p.delta_s[1] + h) : 0.f,
                                p.delta_bias ? __ldg(p.delta_bias + h) : 0.f, p.delta ? __ldg(p.A + h) : 0.f,
                                value<DT>(p.beta + t * p.beta_s[0] + b * p.beta_s[1] + h));
            const float l = fminf(fmaxf(gate.log2a, -255.f), 255.f), hi = rintf(l * 512.f) * (1.f / 512.f);
            sh.ch[tid] = hi, sh.cl[tid] = l - hi, sh.b[tid] = gate.b;
        }
        __syncthreads();
        if (warp < 2) {
            float *c = warp == 0 ? sh.ch : sh.cl;
            const float x = c[2 * lane], y = c[2 * lane + 1] + x;
            float s = y;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const float o = __shfl_up_sync(0xFFFFFFFFu, s, d);
                if (lane >= d)
                    s += o;
            }
            const float o = __shfl_up_sync(0xFFFFFFFFu, s, 1), before = lane > 0 ? o : 0.f;
            c[2 * lane] = before + x;
            c[2 * lane + 1] = before + y;
        }
        __syncthreads();
        for (int e = tid; e < kC * kC; e += kThreads) {
            const int t = e / kC, i = e % kC;
            const float D = i <= t ? ex2(fminf((sh.ch[t] - sh.ch[i]) + (sh.cl[t] - sh.cl[i]), 127.f)) : 0.f;
            sh.L[t][i] = i < t ? sh.b[t] * D * sh.kk[t][i] : 0.f;
            sh.P[t][i] = i <= t ? D * sh.qk[t][i] : 0.f;
            sh.T[t][i] = 0.f;
        }
        __syncthreads();
        if (warp < 4 && lane < 16) {         // the diagonal blocks, a column to a thread
            float x[16];
            const int o = 16 * warp;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = i == lane ? 1.f : 0.f;
#pragma unroll
                for (int m = 0; m < i; ++m)
                    s = fmaf(-sh.L[o + i][o + m], x[m], s);
                x[i] = s;
                sh.T[o + i][o + lane] = s;
            }
        }
        __syncthreads();
        // the corners below them, 16 wide and then 32 wide
        small_product<16>(sh.X, 32 * (tid / 128), 0, sh.L, 32 * (tid / 128) + 16, 32 * (tid / 128), sh.T, 32 * (tid / 128), 32 * (tid / 128), 1.f,
                          tid % 128, 128);
        __syncthreads();
        small_product<16>(sh.T, 32 * (tid / 128) + 16, 32 * (tid / 128), sh.T, 32 * (tid / 128) + 16, 32 * (tid / 128) + 16, sh.X, 32 * (tid / 128), 0,
                          -1.f, tid % 128, 128);
        __syncthreads();
        small_product<32>(sh.X, 0, 0, sh.L, 32, 0, sh.T, 0, 0, 1.f, tid, kThreads);
        __syncthreads();
        small_product<32>(sh.T, 32, 0, sh.T, 32, 32, sh.X, 0, 0, -1.f, tid, kThreads);
        __syncthreads();
        {   // P T, four rows and four columns to a thread
            const int r = 4 * (tid / 16), c = 4 * (tid % 16);
            float s[4][4] = {};
            if (c <= r + 3)
                for (int m = c; m < r + 4; m += 4) {
                    float4 x[4], y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = *reinterpret_cast<const float4 *>(&sh.P[r + i][m]), y[i] = *reinterpret_cast<const float4 *>(&sh.T[m + i][c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            s[i][0] = fmaf(xs[k], y[k].x, s[i][0]), s[i][1] = fmaf(xs[k], y[k].y, s[i][1]);
                            s[i][2] = fmaf(xs[k], y[k].z, s[i][2]), s[i][3] = fmaf(xs[k], y[k].w, s[i][3]);
                        }
                    }
                }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4 *>(&sh.X[r + i][c]) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        }
        __syncthreads();
        const int t = tid / 4, part = tid % 4;
        const float2 of_t = store_terms(sh.T[t], out, out + kPanelBytes, t, part);
        const float2 of_p = store_terms(sh.X[t], out + 2 * kPanelBytes, out + 3 * kPanelBytes, t, part);
        if (part == 0) {
            const float ec = ex2(fminf(sh.ch[t] + sh.cl[t], 127.f));
            const float el = ex2(fminf((sh.ch[kC - 1] - sh.ch[t]) + (sh.cl[kC - 1] - sh.cl[t]), 127.f));
            // a row of zeros adds nothing, and must not lower the others' scale
            const float k = sh.lk[t] != 0.f ? sh.fk[t] * inverse_scale(sh.mk[t]) : 0.f, q = sh.fq[t] * p.scale * inverse_scale(sh.mq[t]);
            factors[kFactorB * kC + t] = sh.b[t];
            factors[kFactorX * kC + t] = sh.b[t] * ec * k;
            factors[kFactorU * kC + t] = of_t.x * el * k;
            factors[kFactorQ * kC + t] = ec * q;
            factors[kFactorP * kC + t] = of_p.x;
            factors[kFactorT * kC + t] = of_t.x;
            factors[kFactorScaleK * kC + t] = sh.mk[t];
            factors[kFactorScaleQ * kC + t] = sh.mq[t];
            sh.of_v[t] = fabsf(sh.b[t]);
            sh.of_s[t] = fabsf(sh.b[t]) * ec * sh.lk[t] * sqrtf((float)p.K);      // |S k'| <= sqrt(K) |k'| max |S|
            sh.of_r[t] = of_t.y * el * fabsf(k);
        }
        __syncthreads();
        if (warp < 3) {
            const float *x = warp == 0 ? sh.of_v : warp == 1 ? sh.of_s : sh.of_r;
            float most = fmaxf(x[lane], x[lane + 32]);
#pragma unroll
            for (int d = 16; d > 0; d /= 2)
                most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
            if (lane == 0)
                factors[kFactorEnd * kC + kEndOfV + warp] = most;
        } else if (tid == 96) {
            factors[kFactorEnd * kC + kEndDecay] = ex2(fminf(sh.ch[kC - 1] + sh.cl[kC - 1], 127.f));
        }
    }
}

template <int DT, int KP>
int32_t prepare(const PrepareParams &p, cudaStream_t stream)
{
    constexpr int bytes = (int)sizeof(PrepareShared<KP>);
    if (cudaFuncSetAttribute(delta_prepare_kernel<DT, KP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return kErrCuda;
    return launch(delta_prepare_kernel<DT, KP>, dim3((unsigned)(p.chunks * p.d.B * p.d.G)), kThreads, bytes, stream, p);
}

}  // namespace

int32_t launch_delta_prepare(const mcc1d_delta_args &a, uint8_t *prepared, cudaStream_t stream)
{
    PrepareParams p = {};
    p.d = delta_params(a);
    p.out = prepared, p.chunks = (a.S + kChunk - 1) / kChunk;
    if (a.dtype == 0)
        return a.K <= 64 ? prepare<0, 64>(p, stream) : prepare<0, 128>(p, stream);
    return a.K <= 64 ? prepare<1, 64>(p, stream) : prepare<1, 128>(p, stream);
}

}  // namespace mcc1d
