// tmap.cu -- host-side TMA tensor-map encoding for bf16 tiles with 64- or
// 128-byte swizzle (cuTensorMapEncodeTiled, resolved through the runtime's driver
// entry point so that the library needs no link-time libcuda).
#include <mutex>

#include "kernels.h"

namespace moe {

namespace {
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}
}  // namespace

bool tensor_maps_available() { return encode_fn() != nullptr; }

namespace {
CUtensorMapSwizzle swizzle_for(uint32_t bytes) {
    return bytes == 0 ? CU_TENSOR_MAP_SWIZZLE_NONE
                      : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
}
}  // namespace

bool tensor_map_2d_bf16(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols,
                        uint32_t box_cols, uint32_t box_rows, uint32_t swizzle_bytes) {
    if (!encode_fn()) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * 2};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims,
                       strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle_for(swizzle_bytes), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tensor_map_3d_bf16(CUtensorMap *m, const void *base, uint64_t n_mat, uint64_t rows,
                        uint64_t cols, uint32_t box_cols, uint32_t box_rows,
                        uint32_t swizzle_bytes) {
    if (!encode_fn()) return false;
    const cuuint64_t dims[3] = {cols, rows, n_mat};
    const cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
    const cuuint32_t box[3] = {box_cols, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                       strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle_for(swizzle_bytes), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tensor_map_2d_u8(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols,
                      uint32_t box_cols, uint32_t box_rows, uint32_t swizzle_bytes) {
    if (!encode_fn()) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols};
    const cuuint32_t box[2] = {box_cols, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims,
                       strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle_for(swizzle_bytes), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tensor_map_3d_u8(CUtensorMap *m, const void *base, uint64_t n_mat, uint64_t rows,
                      uint64_t cols, uint32_t box_cols, uint32_t box_rows,
                      uint32_t swizzle_bytes) {
    if (!encode_fn()) return false;
    const cuuint64_t dims[3] = {cols, rows, n_mat};
    const cuuint64_t strides[2] = {cols, rows * cols};
    const cuuint32_t box[3] = {box_cols, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims,
                       strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle_for(swizzle_bytes), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tensor_map_pair_u8(CUtensorMap *m, const void *first, uint64_t gap, uint64_t n_mat,
                        uint64_t rows, uint64_t cols, uint32_t box_cols, uint32_t group,
                        uint32_t box_groups) {
    if (!encode_fn()) return false;
    const cuuint64_t dims[5] = {cols, group, 2, rows / group, n_mat};
    const cuuint64_t strides[4] = {cols, gap, group * cols, rows * cols};
    const cuuint32_t box[5] = {box_cols, group, 2, box_groups, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(first), dims,
                       strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       swizzle_for(128), CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe
