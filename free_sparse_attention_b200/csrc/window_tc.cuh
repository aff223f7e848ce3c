// TMA access to strided [B, heads, N, d] tensors, shared by the window attention kernels.
#pragma once

#include "tc_common.cuh"
#include "window.cuh"

#include <cstddef>

namespace scope {

// 4-D tile (64 channels x rows of one head) of a strided [B, heads, N, d] tensor.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap *tm, int c, int n, int h, int b, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c), "r"(n), "r"(h), "r"(b), "r"(bar)
        : "memory");
}

// [B, heads, N, d] bf16 with strides: tiles of 64 channels x `rows` tokens of one head,
// 128-byte swizzle, zeros past the last token.
inline bool rows_map(CUtensorMap *m, const void *base, const WinLayout &l, int B, int heads, int N, int d, int rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)heads, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)l.n * 2, (cuuint64_t)l.h * 2, (cuuint64_t)l.b * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace scope
