// kv_maps.h -- tensor maps of the cache's pages and of the drafted rows, for the
// kernels that load them through TMA (host side).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "kv_tc.cuh"

namespace gdn {

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, found once (the library links no driver library); NULL where there is none.
inline Encode encoder() {
    static const Encode fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<Encode>(p);
    }();
    return fn;
}

// 16-bit rows [n3][n2][n1][d] with strides s3, s2, s1 (elements), boxes of `rows2` x `rows` x 64 elements in
// the 128-byte swizzle; past the ends zeros are read. Rows that share memory (a stride of zero) or run
// backwards are not described by a map: false, as where the driver refuses one.
inline bool encode(CUtensorMap& m, int dtype, const void* p, int d, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t n3,
            int64_t s3, int rows, int rows2 = 1) {
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)n1, (cuuint64_t)n2, (cuuint64_t)n3};
    if ((n1 > 1 && s1 < 1) || (n2 > 1 && s2 < 1) || (n3 > 1 && s3 < 1)) return false;
    const auto bytes = [&](int64_t n, int64_t st) { return (cuuint64_t)(n > 1 ? st : d) * 2; };  // of one: any
    const cuuint64_t strides[3] = {bytes(n1, s1), bytes(n2, s2), bytes(n3, s3)};
    const cuuint32_t box[4] = {kvt::BOX, (cuuint32_t)rows, (cuuint32_t)rows2, 1}, unit[4] = {1, 1, 1, 1};
    return encoder()(&m, dtype == GDN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                     const_cast<void*>(p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int boxes_of(int d) { return (d + kvt::BOX - 1) / kvt::BOX; }

// Keys of one box: the largest power of two that divides the page (so that a box lies in one page), up
// to the tile; 0 where it is under the swizzle's eight rows.
inline int box_rows_of(int page_size) {
    int r = page_size & -page_size;
    if (r > kvt::KT) r = kvt::KT;
    return r >= 8 ? r : 0;
}

}  // namespace gdn
