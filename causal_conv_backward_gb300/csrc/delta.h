// delta.h - host-side entry of the gated delta rule's kernels: plans
// (workspace layout) and launches. Arguments have been validated by the caller
// (delta_api.cpp).
#pragma once

#include <cuda_runtime_api.h>
#include <stdint.h>

#include "mcc1d_delta.h"

namespace mcc1d {

constexpr int kMaxKey = 128, kMaxValue = 1024;
constexpr int kChunk = 64;                 // tokens whose products are taken together
constexpr double kUnitEps = 1e-6;          // under the root of |q|^2, |k|^2

// What a pass over the tokens writes down for the gradients: u(t) or du(t)
// [S,B,H,Vp], and the states (or their gradients) at chunks' ends
// [chunks][B H][K,Vp].
struct DeltaKept {
    float *u, *states;
    int32_t Vp;                            // V to a multiple of four
};

// Workspace of the backward, in bytes from its start.
struct DeltaBwdPlan {
    bool tokens;                           // token by token
    int64_t chunks;                        // ceil(S / kChunk)
    int32_t Vp;
    uint64_t off_u, off_du;                // u(t) and its gradient
    uint64_t off_s, off_g;                 // states before each chunk, gradients of those after it
    uint64_t off_sums;                     // grad_A, grad_delta_bias of each (chunk, sequence): [2][chunks B][H]
    uint64_t off_forward, off_grads;       // the forward's own, gradients at the ends of segments
    uint64_t bytes;
};
DeltaBwdPlan delta_bwd_plan(const mcc1d_delta_bwd_args &a);

// What the products of a chunk need beside q, k and v, for each (b, h, chunk):
// T and P T as fp16 terms in the panels that the tensor cores read, the factors
// of its tokens, and in the row kFactorEnd what is one value (delta_prepare.cu).
// The forward's: T, factors, and for y P T; behind it the backward's: T, P T, factors.
constexpr int kPanelBytes = kChunk * 128, kFactorRows = 12, kFactorBytes = kFactorRows * kChunk * 4;
constexpr int kAtT = 0, kAtTLo = kPanelBytes, kAtFactors = 2 * kPanelBytes, kStatesBytes = kAtFactors + kFactorBytes, kAtPT = kStatesBytes,
              kAtPTLo = kAtPT + kPanelBytes, kForwardBytes = kAtPTLo + kPanelBytes;
constexpr int kAtBackT = 0, kAtBackTLo = kPanelBytes, kAtBackPT = 2 * kPanelBytes, kAtBackPTLo = 3 * kPanelBytes, kAtBackFactors = 4 * kPanelBytes,
              kBackBytes = kAtBackFactors + kFactorBytes;
enum { kFactorB, kFactorX, kFactorU, kFactorQ, kFactorP, kFactorScaleK, kFactorScaleQ, kFactorEnd,
       kFactorT, kFactorXY, kFactorY, kFactors };
static_assert(kFactors <= kFactorRows && kAtPT % 1024 == 0 && kForwardBytes % 1024 == 0 && kBackBytes % 1024 == 0, "panels on 1024 bytes");
// In that row: how many tokens come before the first whose k or gates are not
// finite; the chunk's decay; what bounds the state's part of a row's R, U (of R), and
// backwards what the state's gradient is multiplied with first, its part and grad_y's
// of du as an operand; the largest factor of q.
enum { kEndGood, kEndDecay, kEndOfState, kEndOfR, kEndOfGrad, kEndDuOfGrad, kEndDuOfY, kEndMostQ };
constexpr int kBothBytes = kStatesBytes + kBackBytes;        // of a chunk in a backward; kForwardBytes in a forward

struct DeltaPlan {
    bool tokens;                           // token by token, no workspace
    int64_t chunks;                        // ceil(S / kChunk)
    int32_t segments;                      // of the time axis that are taken at once
    uint64_t off_prepared, off_states, off_turns, bytes;
};
DeltaPlan delta_plan(const mcc1d_delta_args &a, bool back);       // back: of a backward's forward

int32_t launch_delta(const mcc1d_delta_args &a, void *workspace, cudaStream_t stream);
int32_t launch_delta_prepare(const mcc1d_delta_args &a, uint8_t *prepared, bool back, cudaStream_t stream);
int32_t launch_delta_chunks_bwd(const mcc1d_delta_bwd_args &a, const DeltaPlan &plan, const uint8_t *forward, float *grads, const DeltaKept &kept,
                                cudaStream_t stream);
int32_t launch_delta_chunks(const mcc1d_delta_args &a, const DeltaPlan &plan, uint8_t *workspace, const DeltaKept &kept, cudaStream_t stream);
// States at the ends of segments, from empty states, become those with which the
// next segments begin: states [segments-1][heads][V,K] in place, s(j) = s(j-1)
// turns(j) + s(j), turns [segments-1][heads][K,K] from j = 1 on. `back`: the
// segments from the last one, with the turns transposed. (delta_join.cu)
int32_t launch_delta_join(float *states, const float *turns, int64_t heads, int32_t V, int32_t K, int32_t segments, bool back, cudaStream_t stream);
int32_t launch_delta_bwd(const mcc1d_delta_bwd_args &a, void *workspace, cudaStream_t stream);
int32_t launch_delta_step(const mcc1d_delta_step_args &a, cudaStream_t stream);

// Token by token (delta_tokens.cu): the forward, with u(t) and the states at
// chunk starts written down where the pointers are given; and the states'
// gradients backwards, with du(t), those at chunk ends and grad_v.
int32_t launch_delta_tokens(const mcc1d_delta_args &a, const DeltaKept &kept, cudaStream_t stream);
int32_t launch_delta_tokens_bwd(const mcc1d_delta_bwd_args &a, const DeltaKept &kept, cudaStream_t stream);

}  // namespace mcc1d
