// Host-side creation of TMA tensor maps (cuTensorMapEncodeTiled through the
// runtime's driver entry point, so the library links no libcuda directly).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ldn {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled_fn()
{
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn = (EncodeTiledFn)p;
    }
    return fn;
}

// 4-D bf16 tensor [d3][d2][d1][d0] (d0 contiguous) viewed through a box of
// {box0, 1, box2, 1} with 128-byte swizzle.  For the [B][T][H][d] activations
// of this library: d0 = d, d1 = H, d2 = T, d3 = B; rows past T read as zero.
inline bool make_tmap_bf16_4d(CUtensorMap *map, const void *base, uint64_t d0, uint64_t d1, uint64_t d2,
                              uint64_t d3, uint32_t box0, uint32_t box2)
{
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t dims[4] = {d0, d1, d2, d3};
    const cuuint64_t strides[3] = {d0 * 2, d0 * d1 * 2, d0 * d1 * d2 * 2};   // bytes, dims 1..3
    const cuuint32_t box[4] = {box0, 1, box2, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `planes` matrices [rows][width] of 16-bit (bf16) or 8-bit elements, rows `ld` and planes
// `plane` elements apart (multiples of 16 bytes), viewed through boxes of `box` rows of 128 bytes
// with 128-byte swizzle.  What lies past a row's width or the rows reads as zero.
inline bool make_tmap_rows(CUtensorMap *map, const void *base, uint64_t width, uint64_t rows, uint64_t planes,
                           uint64_t ld, uint64_t plane, uint32_t box, bool bytes)
{
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const uint64_t es = bytes ? 1 : 2;
    const cuuint64_t dims[3] = {width, rows, planes};
    const cuuint64_t strides[2] = {ld * es, plane * es};
    const cuuint32_t boxes[3] = {(cuuint32_t)(128 / es), box, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void *>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A matrix [rows][width] of fp32, contiguous, viewed through boxes of `box` rows of 128, unswizzled.
inline bool make_tmap_f32(CUtensorMap *map, const void *base, uint64_t width, uint64_t rows, uint32_t box)
{
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {width, rows, 1};
    const cuuint64_t strides[2] = {width * 4, width * 4};
    const cuuint32_t boxes[3] = {128, box, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(base), dims, strides, boxes, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ldn
