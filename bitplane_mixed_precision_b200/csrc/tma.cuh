// Tiled TMA loads: tensor maps made on the host, and the loads into this CTA's shared memory.
#pragma once

#include <cuda.h>

#include "common.h"
#include "pipe.cuh"

namespace pmoe {
namespace tma {

// Map of a row-major tensor of `rank` dimensions (innermost first; strides in bytes of dimensions 1..) whose
// box's rows are 128 bytes, stored with the 128-byte swizzle (16-byte chunk ^= row % 8). Elements outside the
// tensor read as zeros.
// Misses fetch 256 bytes into the L2, half of them the next box's along a row: the 2048-token q8 down products over
// 512 experts took 357 us against 393 with 128 bytes, or none, of promotion.
inline pmoe_status make_map(CUtensorMap *map, int elem_bytes, int rank, const void *base, const uint64_t *dims,
                            const uint64_t *strides, const uint32_t *box)
{
    using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found);
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(f) : nullptr;
    }();
    if (!encode)
        return cuda_status(cudaErrorNotSupported);
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    const CUresult r = encode(map, elem_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                              (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, ones,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PMOE_OK : cuda_status(cudaErrorInvalidValue);
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Loads into this CTA's shared memory, completed in bytes on bar.
__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
                 "[%4];" ::"r"(pipe::smem_u32(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(pipe::smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
                 "%4, %5}], [%6];" ::"r"(pipe::smem_u32(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(pipe::smem_u32(bar))
                 : "memory");
}

} // namespace tma
} // namespace pmoe
