// tensor_maps.cuh -- tensor maps of the paged cache for the tcgen05 kernels.
#pragma once
#include "cache_host.cuh"
#include "tree_attention_tc.cuh"

namespace {

using TensorMapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

TensorMapEncode tensor_map_encode() {
    static const TensorMapEncode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<TensorMapEncode>(f);
    }();
    return encode;
}

// Boxes for the cache's blocks, if they fill tiles of 128 rows evenly; false:
// they do not, or the pool is outside what a tensor map can say.
bool make_pool_maps(const KvView& kv, TcMaps& maps) {
    const int bs = static_cast<int>(kv.block.d);
    if (bs % 8 || (128 % bs && bs % 128) || kv.blocks < 1 || kv.block_stride >= (1ll << 38)) return false;
    const TensorMapEncode encode = tensor_map_encode();
    if (!encode) return false;
    maps.rows = bs < 128 ? bs : 128;
    const int64_t head = static_cast<int64_t>(bs) * kv.dim;
    const int64_t flat = kv.block_stride / head;
    maps.flat = kv.dim == 128 && kv.block_stride % head == 0 && flat * (kv.blocks + 1) < INT32_MAX ? static_cast<int>(flat) : 0;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.dim), static_cast<cuuint64_t>(bs),
                                static_cast<cuuint64_t>(kv.heads), static_cast<cuuint64_t>(kv.blocks)};
    const cuuint64_t strides[3] = {dims[0] * 2, dims[0] * dims[1] * 2, static_cast<cuuint64_t>(kv.block_stride) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(maps.rows), 1, 1}, ones[5] = {1, 1, 1, 1, 1};
    const cuuint64_t flat_dims[5] = {64, 8, 2, dims[1] / 8, static_cast<cuuint64_t>(flat * (kv.blocks - 1) + kv.heads)};
    const cuuint64_t flat_strides[4] = {256, 128, 2048, static_cast<cuuint64_t>(head) * 2};
    const cuuint32_t flat_box[5] = {64, 8, 2, static_cast<cuuint32_t>(maps.rows / 8), 1};
    for (int i = 0; i < 2; ++i)
        if (encode(i ? &maps.v : &maps.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, maps.flat ? 5 : 4, i ? kv.v : kv.k,
                   maps.flat ? flat_dims : dims, maps.flat ? flat_strides : strides, maps.flat ? flat_box : box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    return true;
}

}  // namespace
