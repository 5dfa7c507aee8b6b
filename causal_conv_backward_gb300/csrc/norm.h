// norm.h - host-side entry of the gated norm's and the residual norm's kernels.
// Arguments have been validated by the caller (norm_api.cpp).
#pragma once

#include <cuda_runtime_api.h>
#include <stdint.h>

#include "mcc1d_norm.h"

namespace mcc1d {

constexpr int64_t kMaxNormRow = 16384;

// Column sums over the rows go through partial sums of each block:
// [sums][blocks][columns] fp32 in the workspace.
constexpr int kGatedThreads = 768, kResidualThreads = 512;      // of a backward, on an SM: what its registers allow
int64_t norm_bwd_blocks(int64_t rows, int64_t columns, bool vectors, int threads);
bool gated_norm_vectors(const mcc1d_gated_norm_bwd_args &a);
bool residual_norm_vectors(const mcc1d_residual_norm_bwd_args &a);
inline uint64_t norm_bwd_bytes(int64_t blocks, int64_t columns, int sums) { return 4ull * sums * blocks * columns; }

int32_t launch_gated_norm(const mcc1d_gated_norm_args &a, cudaStream_t stream);
int32_t launch_gated_norm_bwd(const mcc1d_gated_norm_bwd_args &a, float *workspace, cudaStream_t stream);
int32_t launch_residual_norm(const mcc1d_residual_norm_args &a, cudaStream_t stream);
int32_t launch_residual_norm_bwd(const mcc1d_residual_norm_bwd_args &a, float *workspace, cudaStream_t stream);

// out[c] = sum of part[p][c] over p, rounded to dtype 0, 1 or (2) kept fp32;
// null outputs are left out. In norm_gated.cu.
struct ColumnSums {
    const float *part[3];
    void *out[3];
    int32_t type[3];
};
int32_t launch_column_sums(const ColumnSums &s, int64_t parts, int64_t columns, int sums, cudaStream_t stream);

}  // namespace mcc1d
