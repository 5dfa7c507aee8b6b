// tensor_map.cpp - tile descriptors by the encoder that libcuda exports.
#include "tensor_map.h"

#include <cuda_runtime_api.h>

namespace mcc1d {

namespace {

typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                           const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder()
{
    static const Encode fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<Encode>(p);
    }();
    return fn;
}

}  // namespace

bool token_tiles(CUtensorMap *map, const void *at, int64_t S, int64_t B, int64_t heads, int64_t n, const int64_t (&strides)[3], bool panels)
{
    if (((uintptr_t)at & 15u) || n % 8)
        return false;
    const cuuint64_t dims[4] = {(cuuint64_t)n, (cuuint64_t)S, (cuuint64_t)heads, (cuuint64_t)B};
    const int64_t of[3] = {strides[0], strides[2], strides[1]};
    cuuint64_t steps[3];
    for (int i = 0; i < 3; ++i) {
        const bool one = dims[i + 1] == 1;          // never stepped along
        if (!one && (of[i] <= 0 || of[i] % 8 || of[i] >= ((int64_t)1 << 38)))
            return false;
        steps[i] = one ? 16 : 2 * (cuuint64_t)of[i];
    }
    const cuuint32_t box[4] = {64, 64, 1, 1}, every[4] = {1, 1, 1, 1};
    const Encode encode = encoder();
    return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(at), dims, steps, box, every, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            panels ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mcc1d
