// ssm.h - host-side entry of the short convolution's and the selective scan's
// kernels: their plans (workspace layout, time chunks) and launches.
// Arguments have been validated by the caller (ssm_api.cpp).
#pragma once

#include <cuda_runtime_api.h>
#include <stdint.h>

#include "mcc1d_ssm.h"

namespace mcc1d {

constexpr int kMaxStates = 64;   // N of the selective scan

// ------------------------------------------------------------------ short convolution
// Rows of one (sequence, 8 warps x L rows) block of the backward, whose
// gradWeight and gradBias partials go to the workspace: [parts][W+1][H] fp32.
struct ConvBwdPlan {
    int32_t L;            // rows per warp
    int64_t supers;       // blocks of 8 L rows per sequence
    int64_t parts;        // B * supers
    uint64_t bytes;
};
ConvBwdPlan conv_bwd_plan(const mcc1d_short_conv_bwd_args &a);

int32_t launch_short_conv(const mcc1d_short_conv_args &a, cudaStream_t stream);
int32_t launch_short_conv_bwd(const mcc1d_short_conv_bwd_args &a, void *workspace, cudaStream_t stream);
int32_t launch_short_conv_step(const mcc1d_short_conv_step_args &a, cudaStream_t stream);

// ------------------------------------------------------------------ selective scan
// How blocks cover the channels.
struct ScanGrid {
    int64_t blocks;           // over all groups
    int32_t blocks_per_group;
};

// A channel's N states are spread over NL = 1, 2, 4, 8 or 16 lanes of a warp,
// four to a lane (NP = 4 NL >= N, padded with zeros). Blocks walk one time
// chunk of their channels in tiles of TT rows.
struct ScanPlan {
    int32_t nl, np, tt;
    int64_t tiles;            // ceil(S / tt)
    int64_t tiles_per_chunk;
    int64_t chunks;
    uint64_t off_e, off_r, off_dt, off_cp, off_cpdt, off_ga, off_gd, off_bc;   // workspace, in bytes
    uint64_t bytes;
    int64_t most_blocks;      // of the largest grid
    ScanGrid grid;            // of the passes
};
ScanPlan scan_plan(const mcc1d_scan_args &a);
ScanPlan scan_bwd_plan(const mcc1d_scan_bwd_args &a);

int32_t launch_scan(const mcc1d_scan_args &a, const ScanPlan &p, void *workspace, cudaStream_t stream);
int32_t launch_scan_bwd(const mcc1d_scan_bwd_args &a, const ScanPlan &p, void *workspace, cudaStream_t stream);
int32_t launch_scan_step(const mcc1d_scan_step_args &a, cudaStream_t stream);

}  // namespace mcc1d
