// tensor_map.h -- TMA descriptors of cache and query views (host side).
#pragma once

#include <cstdint>

#include <cuda.h>

#include "pages.h"
#include "serving.h"

namespace splitzip {

// A [batch, tokens, heads, D] view as a tensor map of boxes of 64 16-bit values in
// swizzled rows (or whole rows of 8-bit ones as they are or, swizzle8, by their length), `box_heads` heads and
// `box_tokens` tokens.  A dimension of length 1 gets some valid stride; a
// batch stride of 0 becomes length 1 (one_batch: its coordinate is always 0).
inline bool make_map(CUtensorMap& map, const splitzip_view& v, uint32_t elem, uint32_t dim, uint32_t heads, uint32_t tokens, uint32_t batch,
              uint32_t box_heads, uint32_t box_tokens, bool heads_first, uint32_t* one_batch, bool swizzle8 = false) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    if (!encode) return false;
    const uint64_t any = elem * dim;
    *one_batch = batch == 1 || v.stride_b == 0;
    const uint64_t nb = *one_batch ? 1 : batch;
    const uint64_t sh = heads > 1 ? elem * (uint64_t)v.stride_h : any, st = tokens > 1 ? elem * (uint64_t)v.stride_t : any;
    const uint64_t sb = *one_batch ? any : elem * (uint64_t)v.stride_b;
    const cuuint64_t sizes[4] = {dim, heads_first ? heads : tokens, heads_first ? tokens : heads, nb};
    const cuuint64_t strides[3] = {heads_first ? sh : st, heads_first ? st : sh, sb};
    const cuuint32_t box[4] = {elem == 1 ? dim : 64, heads_first ? box_heads : box_tokens, heads_first ? box_tokens : box_heads, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const CUtensorMapSwizzle swizzle = elem == 2    ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : !swizzle8  ? CU_TENSOR_MAP_SWIZZLE_NONE
                                       : dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : dim == 64  ? CU_TENSOR_MAP_SWIZZLE_64B
                                                    : CU_TENSOR_MAP_SWIZZLE_32B;
    return encode(&map, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.data, sizes, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A pool's keys or values as a map of boxes of `box` slots of a page and head, at
// (value or byte, slot, head, page); rows of bytes are swizzled by their length.
inline bool page_map(CUtensorMap& map, const splitzip_pool& pool, const splitzip_page_rows& rows, uint32_t box) {
    uint32_t one;
    const bool bytes = pool.format >= SPLITZIP_FORMAT_E5M2 && pool.format <= SPLITZIP_FORMAT_E2M1;  // else 16 bits, of which a copy takes no notice
    const uint32_t elem = bytes ? 1 : 2, dim = pool.format == SPLITZIP_FORMAT_E2M1 ? pool.head_dim / 2 : pool.head_dim;
    return make_map(map, {rows.data, rows.stride_p, rows.stride_t, rows.stride_h}, elem, dim, pool.kv_heads, pool.page_tokens, pool.pages, 1, box,
                    false, &one, true);
}

}  // namespace splitzip
