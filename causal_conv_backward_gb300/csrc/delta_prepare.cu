// delta_prepare.cu - a chunk's products of tokens with tokens.
//
// With c(t) the running sum of log a, D(t,i) = exp(c(t) - c(i)):
//   L(t,i) = b(t) D (k'(t).k'(i)), i < t;   P(t,i) = D (q'(t).k'(i)), i <= t
//   T = (I + L)^-1,   so that U = T R for R = b (V - e^c K' S^T),  and P U = (P T) R
// T and P T leave as two fp16 terms each (22 bits), rows scaled by powers of two,
// in the layout that delta_chunks.cu multiplies from, for an R that a token's growth
// has been taken out of (growth_of). All paths from i to t pass the same decays, so that
// powers of two by token change those of T and P T value by value.
//
// k'.k' and q'.k' are taken of the 16-bit tensors themselves on the tensor cores
// (their products are exact in fp32) and scaled afterwards. The inverse is that
// of the 16-wide diagonal blocks by substitution, joined twice:
// [[A,0],[C,B]]^-1 = [[A',0],[-B' C A',B']].
//
// A block has one chunk of one head, three blocks an SM: 2048 tokens of 8 x 16
// heads of K = 128 take 196 us with what a backward needs, where their 360 MB would
// take 53 (the second panels' stores 25 us of it, their columns' scales 14). The
// dependent steps of the inverse and the barriers between its parts bound it, which
// three blocks hide from one another in part.
#include "delta_common.cuh"
#include "tensor_core.cuh"

namespace mcc1d {

namespace {

constexpr int kC = kChunk, kThreads = 256, kRow = kC + 4;

struct PrepareParams {
    DeltaParams d;
    uint8_t *out;
    int64_t chunks;
    bool vectors_q, vectors_k;
};

// Rows of 16-bit values eight longer, so that eight of them start on different
// banks. What the tokens' rows take is T and X later on.
template <int KP>
struct PrepareShared {
    static constexpr int RS = KP + 8;
    union {
        uint16_t qk[2][kC][RS];
        struct {
            float T[kC][kRow], X[kC][kRow];
        };
    };
    float L[kC][kRow], P[kC][kRow];
    float ch[kC], cl[kC], rest[kC], grown[kC], b[kC], f[2][kC], m[2][kC], lk[kC], late[kC], whole[kC], of_t[kC], sum_t[kC], of_p[kC], ends[4][8];
    bool zero_q[kC];
    uint32_t bad_gates[2];
    int bad_k[4];
};

template <int DT>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (DT == 0)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A value as two tf32 terms, 22 bits, and their products.
__device__ __forceinline__ void tf32_terms(float x, uint32_t &hi, uint32_t &lo)
{
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(lo) : "f"(x - __uint_as_float(hi)));
}
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four 8 x 8 matrices of 16-bit values, the rows' addresses from eight lanes each.
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
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

// 16 values of row t of a matrix as two panels.
__device__ __forceinline__ void store_terms(const float (&x)[16], float scale, uint8_t *hi, uint8_t *lo, int t, int part)
{
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
}
__device__ __forceinline__ float most_of_warp(float x)
{
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
    return x;
}
// The largest of a row over its four threads, and the sum of all.
__device__ __forceinline__ float most_of_row(const float (&x)[16], float &sum)
{
    float most = 0.f;
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        most = fmaxf(most, fabsf(x[j])), sum += fabsf(x[j]);
#pragma unroll
    for (int d = 1; d < 4; d *= 2)
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d)), sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    return most;
}

// The whole powers of two of e^c, of which T is a quotient.
__device__ __forceinline__ float whole_of(float c) { return fminf(fmaxf(rintf(c), -100.f), 126.f); }
// What is taken out of a token's R and put back by its column of T and P T, as a
// power of two, from the logarithm c of all decays up to it. Two terms hold a row to
// 2^-40 of its largest value, and a token's R has two parts, its value and the
// state's, e^c S k. All of a growth (c > 0), which else only the last tokens would be
// seen of; half of a decay, up to 2^17, so that where values are small both R, which
// falls by the other half, and T keep their bits.
__device__ __forceinline__ float growth_of(float c)
{
    return c > 0.f ? fminf(rintf(c), 126.f) : fmaxf(rintf(0.5f * c), -17.f);
}

template <int DT, int KP, bool BACK>
__global__ void __launch_bounds__(kThreads, 3) mcc1d_delta_prepare_chunk(const __grid_constant__ PrepareParams pp)
{
    extern __shared__ __align__(16) uint8_t raw_shared[];
    typedef PrepareShared<KP> Shared;
    Shared &sh = *reinterpret_cast<Shared *>(raw_shared);
    const DeltaParams &p = pp.d;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int h = blockIdx.x % p.H, b = (blockIdx.x / p.H) % p.B, g = h / (p.H / p.G);
    const int64_t chunk = blockIdx.x / p.H / p.B, t0 = chunk * kC;
    const int64_t length = clamped_length(p.lengths, b, p.S);
    if (length <= t0)
        return;
    const int n = (int)(length - t0 < kC ? length - t0 : kC);
    const int64_t item = (int64_t)b * p.H + h;
    uint8_t *out = pp.out + (item * pp.chunks + chunk) * (BACK ? kBothBytes : kForwardBytes);

    // rows of q and k, all of a thread's loads in flight together
    constexpr int PIECES = KP / 8, STEP = kThreads / PIECES, N = kC / STEP;
    {
        const int piece = tid % PIECES, first = tid / PIECES;
        uint4 x[2][N];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const int64_t step = w ? p.k_s[0] : p.q_s[0];
            const uint16_t *from = w ? p.k + b * p.k_s[1] + g * p.k_s[2] : p.q + b * p.q_s[1] + g * p.q_s[2];
            from += (t0 + first) * step + 8 * piece;
            const bool vectors = w ? pp.vectors_k : pp.vectors_q;
#pragma unroll
            for (int j = 0; j < N; ++j, from += STEP * step) {
                const int live = first + j * STEP < n ? p.K - 8 * piece : 0;
                x[w][j] = make_uint4(0u, 0u, 0u, 0u);
                if (vectors) {
                    if (live > 0)
                        x[w][j] = __ldg(reinterpret_cast<const uint4 *>(from));
                } else {
                    uint32_t *e = reinterpret_cast<uint32_t *>(&x[w][j]);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < live)
                            e[i / 2] |= (uint32_t)__ldg(from + i) << (16 * (i % 2));
                }
            }
        }
        // gates, and the running sum of log2 a in two parts whose differences are
        // exact in the first: multiples of 2^-9 below 2^14
        if (tid < kC) {
            const int64_t t = t0 + tid;
            Gates gate = {0.f, 0.f, 0.f, 0.f};
            if (tid < n)
                gate = gates_of(p.flags, p.delta != nullptr, p.delta ? value<DT>(p.delta + t * p.delta_s[0] + b * p.delta_s[1] + h) : 0.f,
                                p.delta_bias ? __ldg(p.delta_bias + h) : 0.f, p.delta ? __ldg(p.A + h) : 0.f,
                                value<DT>(p.beta + t * p.beta_s[0] + b * p.beta_s[1] + h));
            const float l = held_log2(gate.log2a), hi = rintf(l * 512.f) * (1.f / 512.f);
            sh.ch[tid] = hi, sh.cl[tid] = l - hi, sh.b[tid] = gate.b;
            const uint32_t bad = __ballot_sync(0xFFFFFFFFu, !(l == l && fabsf(gate.b) < INFINITY));
            if (lane == 0)
                sh.bad_gates[warp] = bad;
        }
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int j = 0; j < N; ++j)
                *reinterpret_cast<uint4 *>(&sh.qk[w][first + j * STEP][8 * piece]) = x[w][j];
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
    {   // lengths, and the scale that makes rows of about one size of them in fp16, without loss: two threads to a row
        const int w = tid / 128, t = tid % 128 / 2, half = tid % 2;
        float sum = 0.f, most = 0.f;
#pragma unroll
        for (int j = 0; j < KP / 16; ++j) {
            const uint4 v = *reinterpret_cast<const uint4 *>(&sh.qk[w][t][(2 * j + half) * 8]);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = unpack2<DT>(u[e]);
                sum = fmaf(x.x, x.x, fmaf(x.y, x.y, sum));
                most = fmaxf(most, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
        }
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        const uint32_t bad = __ballot_sync(0xFFFFFFFFu, !(sum == sum && most < INFINITY));
        if (w == 1 && lane == 0)
            sh.bad_k[warp - 4] = bad ? 16 * (warp - 4) + (__ffs(bad) - 1) / 2 : kC;
        if (half == 0) {
            const float f = unit_factor(p.flags, sum);
            sh.f[w][t] = f, sh.m[w][t] = scale_for(most);
            if (w == 1)
                sh.lk[t] = sqrtf(sum) * f;
            else
                sh.zero_q[t] = most == 0.f;
        }
    }
    __syncthreads();
    // From the first token on whose k or gates are not finite all outputs are NaN, and
    // so is the state; the tokens before it know nothing of them: no zero of T meets
    // them. (Gradients do not keep to that: theirs are NaN for the whole chunk.)
    int good = min(min(sh.bad_k[0], sh.bad_k[1]), min(sh.bad_k[2], sh.bad_k[3]));
    if (sh.bad_gates[0] | sh.bad_gates[1])
        good = min(good, sh.bad_gates[0] ? __ffs(sh.bad_gates[0]) - 1 : 31 + __ffs(sh.bad_gates[1]));
    if (tid < kC) {
        const float growth = growth_of(sh.ch[tid] + sh.cl[tid]);
        sh.rest[tid] = sh.ch[tid] - growth, sh.grown[tid] = ex2(growth);
    }
    {   // 16 rows and 32 columns of both products to a warp
        const int r0 = 16 * (warp % 4), c0 = 32 * (warp / 4), row = lane / 4, col = 2 * (lane % 4);
        float kk[4][4] = {}, qk[4][4] = {};
        if (c0 <= r0 + 15) {
            constexpr int RS = Shared::RS;
            const uint32_t q = smem_u32(&sh.qk[0][r0 + lane % 16][8 * (lane / 16)]), k = q + kC * RS * 2;
            const uint32_t c = smem_u32(&sh.qk[1][c0 + lane % 8 + 8 * (lane / 16)][8 * (lane / 8 % 2)]);
#pragma unroll
            for (int at = 0; at < KP; at += 16) {
                uint32_t aq[4], ak[4], x[4], y[4];
                load_matrices(aq, q + 2 * at);
                load_matrices(ak, k + 2 * at);
                load_matrices(x, c + 2 * at);
                mma16816<DT>(kk[0], ak, x[0], x[1]), mma16816<DT>(kk[1], ak, x[2], x[3]);
                mma16816<DT>(qk[0], aq, x[0], x[1]), mma16816<DT>(qk[1], aq, x[2], x[3]);
                if (c0 + 16 <= r0) {
                    load_matrices(y, c + 2 * at + 16 * RS * 2);
                    mma16816<DT>(kk[2], ak, y[0], y[1]), mma16816<DT>(kk[3], ak, y[2], y[3]);
                    mma16816<DT>(qk[2], aq, y[0], y[1]), mma16816<DT>(qk[3], aq, y[2], y[3]);
                }
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int t = r0 + row + 8 * half;
            const float th = sh.ch[t], tl = sh.cl[t], lt = sh.b[t] * sh.f[1][t], pt = p.scale * sh.f[0][t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (c0 + 8 * j > r0 + 15)          // above the diagonal: read by nothing
                    continue;
                float l[2], x[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = c0 + 8 * j + col + e;
                    const float D = i <= t ? ex2_held((th - sh.ch[i]) + (tl - sh.cl[i])) * sh.f[1][i] : 0.f;
                    l[e] = i < t && t < good ? kk[j][2 * half + e] * (D * lt) : 0.f;
                    x[e] = i <= t && t < good ? qk[j][2 * half + e] * (D * pt) : 0.f;
                }
                *reinterpret_cast<float2 *>(&sh.L[t][c0 + 8 * j + col]) = make_float2(l[0], l[1]);
                *reinterpret_cast<float2 *>(&sh.P[t][c0 + 8 * j + col]) = make_float2(x[0], x[1]);
            }
        }
    }
    __syncthreads();
    if (warp >= 4) {                     // zeros beside them, above the diagonal, that the wider products read
        const int e = tid - 128, o = 32 * (e / 64), i = e % 64 / 4, j = 16 + 4 * (e % 4);
        *reinterpret_cast<float4 *>(&sh.T[o + i][o + j]) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else if (lane < 16) {              // the diagonal blocks, a column to a thread
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
    {   // P T on the tensor cores, two tf32 terms to a value: 16 rows and every other
        // eight columns to a warp, tokens from the column's to the row's
        const int r0 = 16 * (warp % 4), row = lane / 4, col = lane % 4;
        float acc[4][4] = {};
        for (int m = 0; m < r0 + 16; m += 8) {
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                tf32_terms(sh.P[r0 + row + 8 * (e % 2)][m + col + 4 * (e / 2)], ah[e], al[e]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = 8 * (2 * j + warp / 4);
                if (c > m)
                    continue;
                uint32_t bh[2], bl[2];
                tf32_terms(sh.T[m + col][c + row], bh[0], bl[0]);
                tf32_terms(sh.T[m + col + 4][c + row], bh[1], bl[1]);
                mma1688(acc[j], ah, bl[0], bl[1]);
                mma1688(acc[j], al, bh[0], bh[1]);
                mma1688(acc[j], ah, bh[0], bh[1]);
            }
        }
        // X holds what the last corner was made of: others are past it
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float2 *>(&sh.X[r0 + row + 8 * e][8 * (2 * j + warp / 4) + 2 * col]) = make_float2(acc[j][2 * e], acc[j][2 * e + 1]);
    }
    __syncthreads();
    // four threads to a row
    {
        const int t = tid / 4, part = tid % 4;
        float x[16];
        const auto row_of = [&](const float (*m)[kRow]) {
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(&m[t][16 * part + j]), f = *reinterpret_cast<const float4 *>(&sh.grown[16 * part + j]);
                x[j] = v.x * f.x, x[j + 1] = v.y * f.y, x[j + 2] = v.z * f.z, x[j + 3] = v.w * f.w;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                x[j] = 16 * part + j <= t ? x[j] : 0.f;       // nothing is written behind the diagonal
        };
        row_of(sh.T);
        float sum, scale = scale_for(most_of_row(x, sum));
        store_terms(x, scale, out + kAtT, out + kAtTLo, t, part);
        if (part == 0)
            sh.of_t[t] = inverse_scale(scale), sh.sum_t[t] = sum;
        if (!BACK) {
            row_of(sh.X);
            scale = scale_for(most_of_row(x, sum));
            store_terms(x, scale, out + kAtPT, out + kAtPTLo, t, part);
            if (part == 0)
                sh.of_p[t] = inverse_scale(scale);
        }
    }
    if (BACK) {
        // T without the decays (G's part passes all of them, whatever token it goes
        // through) and P T; these sum over their rows, so that each column is scaled. What
        // takes a growth out of grad_y's rows (from the token to the end) is put into
        // those of P T, and the decays' powers of two taken out of T, as far as 2^-100.
        float (*most)[kRow] = sh.L, (*scales)[kRow] = sh.L + 8;          // L is not read any more
        const int i = tid % kC, first = 16 * (tid / kC);
        float *late = sh.L[10], *by = sh.L[11], *to = sh.L[12];
        if (tid < kC) {
            const float w = whole_of(sh.ch[tid] + sh.cl[tid]);
            sh.late[tid] = growth_of((sh.ch[kC - 1] - sh.ch[tid]) + (sh.cl[kC - 1] - sh.cl[tid]));
            late[tid] = ex2(sh.late[tid]), sh.whole[tid] = w, by[tid] = ex2(-w), to[tid] = ex2(w);
        }
        __syncthreads();
        {
            float most_t = 0.f, most_p = 0.f;
            if (first + 15 >= i) {
                const float to_i = to[i];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int j = first + e;
                    if (j >= i) {
                        const float v = sh.T[j][i] * by[j] * to_i, w = sh.X[j][i] * late[j];
                        most_t = fmaxf(most_t, fabsf(v)), most_p = fmaxf(most_p, fabsf(w));
                        sh.T[j][i] = v, sh.X[j][i] = w;
                    }
                }
            }
            most[tid / kC][i] = most_t, most[4 + tid / kC][i] = most_p;
        }
        __syncthreads();
        if (tid < 2 * kC) {
            const int w = tid / kC;
            most[4 * w][i] = fmaxf(fmaxf(most[4 * w][i], most[4 * w + 1][i]), fmaxf(most[4 * w + 2][i], most[4 * w + 3][i]));
            scales[w][i] = scale_for(most[4 * w][i]);
        }
        __syncthreads();
        const int t = tid / 4, part = tid % 4;
        uint8_t *back = out + kStatesBytes;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const float (*m)[kRow] = w ? sh.X : sh.T;
            float x[16];
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(&m[t][16 * part + j]), f = *reinterpret_cast<const float4 *>(&scales[w][16 * part + j]);
                x[j] = v.x * f.x, x[j + 1] = v.y * f.y, x[j + 2] = v.z * f.z, x[j + 3] = v.w * f.w;
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                x[j] = 16 * part + j <= t ? x[j] : 0.f;
            store_terms(x, 1.f, back + (w ? kAtBackPT : kAtBackT), back + (w ? kAtBackPTLo : kAtBackTLo), t, part);
        }
    } else {
        __syncthreads();
    }
    // the tokens' factors: two warps the forward's, two the backward's
    if (warp < (BACK ? 4 : 2)) {
        const int t = tid % kC;
        const bool back = warp >= 2;
        const float th = sh.ch[t], tl = sh.cl[t], b = sh.b[t], end = sh.ch[kC - 1] + sh.cl[kC - 1];
        const float none = __uint_as_float(0x7FFFFFFFu);
        const bool there = t < good;
        const float ec = ex2_held(th + tl), decay = good < kC ? none : decay_of(end > 127.f ? 127.f : end);
        // a row of zeros adds nothing, and must not lower the others' scale
        const float k = sh.lk[t] != 0.f ? sh.f[1][t] * inverse_scale(sh.m[1][t]) : 0.f;
        const float q = sh.zero_q[t] ? 0.f : sh.f[0][t] * p.scale * inverse_scale(sh.m[0][t]);
        const float reach = sh.lk[t] * sqrtf((float)p.K);                  // |S k'| <= sqrt(K) |k'| max |S|
        float *to = reinterpret_cast<float *>(out + (back ? kStatesBytes + kAtBackFactors : kAtFactors)) + t;
        to[kFactorScaleK * kC] = sh.m[1][t];
        to[kFactorScaleQ * kC] = sh.m[0][t];
        if (!back) {
            const float rest = ex2_held(sh.rest[t] + tl), el = ex2_held((sh.ch[kC - 1] - th) + (sh.cl[kC - 1] - tl)), of = sh.of_t[t];
            to[kFactorB * kC] = there ? b * ex2(sh.rest[t] - th) : 0.f;
            to[kFactorX * kC] = there ? b * rest * k : 0.f;
            to[kFactorU * kC] = of * el * k;
            to[kFactorT * kC] = there ? of : none;
            if (!BACK) {
                to[kFactorQ * kC] = there ? ec * q : none;
                to[kFactorP * kC] = sh.of_p[t];
            }
            const float most[2] = {most_of_warp(there ? fabsf(b) * rest * reach : 0.f), most_of_warp(sh.sum_t[t] * el * fabsf(k))};
            if (lane == 0)
                sh.ends[warp][0] = most[0], sh.ends[warp][1] = most[1], sh.ends[warp][5] = decay;
        } else {
            const float most_t = sh.L[0][t], of_t = good < kC ? none : inverse_scale(sh.L[8][t]), of_p = good < kC ? none : inverse_scale(sh.L[9][t]), bk = b * k;
            const float fq = ex2_held(th + sh.late[t] + tl) * q, w = sh.whole[t], w_end = sh.whole[kC - 1];
            const float fx = bk * ex2_held(th - w + w_end + tl), fu = ex2_held(((sh.ch[kC - 1] - w_end) - (th - w)) + (sh.cl[kC - 1] - tl));
            to[kFactorB * kC] = b;
            to[kFactorX * kC] = fx * of_t;
            to[kFactorXY * kC] = bk * ec * of_p;
            to[kFactorU * kC] = fu * k;
            to[kFactorT * kC] = ex2_held(w_end - w) * of_t;
            to[kFactorP * kC] = of_p;
            to[kFactorQ * kC] = fq;
            to[kFactorY * kC] = ex2(-sh.late[t]);
            const float most[5] = {most_of_warp(fu * reach), most_of_warp(most_t), most_of_warp(fabsf(fx)), most_of_warp(fabsf(bk) * ec * (kC * sh.L[4][t])),
                                   most_of_warp(fabsf(fq))};
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < 5; ++j)
                    sh.ends[warp][j] = most[j];
        }
    }
    __syncthreads();
    if (tid == 0) {
        const auto most = [&](int w, int j) { return fmaxf(sh.ends[w][j], sh.ends[w + 1][j]); };
        const float decay = sh.ends[0][5];
        float *ends = reinterpret_cast<float *>(out + kAtFactors) + kFactorEnd * kC;
        ends[kEndGood] = (float)good, ends[kEndDecay] = decay, ends[kEndOfState] = most(0, 0), ends[kEndOfR] = most(0, 1);
        if (BACK) {
            ends = reinterpret_cast<float *>(out + kStatesBytes + kAtBackFactors) + kFactorEnd * kC;
            ends[kEndDecay] = decay, ends[kEndOfGrad] = most(2, 0), ends[kEndDuOfGrad] = most(2, 0) * (kC * most(2, 1)) * most(2, 2);
            ends[kEndDuOfY] = most(2, 3), ends[kEndMostQ] = most(2, 4);
        }
    }
}

template <int DT, int KP, bool BACK>
int32_t prepare(const PrepareParams &p, cudaStream_t stream)
{
    constexpr int bytes = (int)sizeof(PrepareShared<KP>);
    if (cudaFuncSetAttribute(mcc1d_delta_prepare_chunk<DT, KP, BACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return kErrCuda;
    return launch(mcc1d_delta_prepare_chunk<DT, KP, BACK>, dim3((unsigned)(p.chunks * p.d.B * p.d.H)), kThreads, bytes, stream, p);
}

}  // namespace

int32_t launch_delta_prepare(const mcc1d_delta_args &a, uint8_t *prepared, bool back, cudaStream_t stream)
{
    PrepareParams p = {};
    p.d = delta_params(a);
    p.out = prepared, p.chunks = (a.S + kChunk - 1) / kChunk;
    p.vectors_q = vectors_for(a.K, (uintptr_t)a.q, a.q_strides[0] | a.q_strides[1] | a.q_strides[2]);
    p.vectors_k = vectors_for(a.K, (uintptr_t)a.k, a.k_strides[0] | a.k_strides[1] | a.k_strides[2]);
    const auto go = [&](auto dt, auto b) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool BACK = decltype(b)::value;
        return a.K <= 64 ? prepare<DT, 64, BACK>(p, stream) : prepare<DT, 128, BACK>(p, stream);
    };
    const auto type = [&](auto b) { return a.dtype == 0 ? go(std::integral_constant<int, 0>(), b) : go(std::integral_constant<int, 1>(), b); };
    return back ? type(std::true_type()) : type(std::false_type());
}

}  // namespace mcc1d
