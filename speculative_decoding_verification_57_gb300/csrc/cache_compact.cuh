// cache_compact.cuh -- the kept path of a verified tree moved together in the
// paged cache, keys and values of every layer in one launch.
//
// Node path[i] goes to the place of node i.  A path is strictly increasing,
// so path[i] >= i: no place is written before it was read if the moves run in
// order of i, and a thread that owns the same 16 bytes of every node can run
// them without a barrier.
#pragma once
#include "kv_cache.cuh"

namespace specv {

constexpr int kCompactThreads = 256;

struct CompactArgs {
    KvView kv;
    const int32_t* path;          // [B, M]
    const int32_t* num_accepted;  // [B]
    int32_t* row_status;
    int64_t layer_stride;  // elements
    int M, layers;
    int vecs;  // 16-byte pieces of a head
    int vec_elems;
};

template <typename T>
__global__ void __launch_bounds__(kCompactThreads) cache_compact_kernel(const CompactArgs c) {
    __shared__ int64_t s_src[32], s_dst[32];
    __shared__ int s_status;
    const int b = blockIdx.x, tid = threadIdx.x;
    const KvView& kv = c.kv;
    const int len = kv.lens[b], n = c.num_accepted[b];
    if (tid < 32) {
        int status = 0;
        if (len != 0) {
            if (n < 0 || n > c.M) status |= KV_ACCEPTED;
            if (len < c.M || !kv.fits(len)) status |= KV_LENGTH;
        }
        int node = -1;
        bool path_ok = true, block_ok = true;
        if (status == 0 && len != 0 && tid < n) {
            node = c.path[static_cast<int64_t>(b) * c.M + tid];
            path_ok = node >= 0 && node < c.M;
        }
        const int before = __shfl_up_sync(0xffffffffu, node, 1);
        if (path_ok && tid > 0 && node >= 0) path_ok = node > before;
        if (!__all_sync(0xffffffffu, path_ok)) status |= KV_PATH;
        if (status == 0 && node >= 0) {
            const int32_t* table = kv.tables + static_cast<int64_t>(b) * kv.max_blocks;
            const int src = len - c.M + node, dst = len - c.M + tid;
            const int ls = kv.block.div(src), ld = kv.block.div(dst);
            const int bs = table[ls], bd = table[ld];
            block_ok = kv.valid(bs) && kv.valid(bd);
            s_src[tid] = kv.at(bs, 0, src - ls * kv.block_size());
            s_dst[tid] = kv.at(bd, 0, dst - ld * kv.block_size());
        }
        if (!__all_sync(0xffffffffu, block_ok)) status |= KV_BLOCK;
        if (tid == 0) {
            s_status = status;
            if (blockIdx.y == 0 && c.row_status) c.row_status[b] = status;
        }
    }
    __syncthreads();
    if (s_status != 0 || len == 0 || n <= 0) return;
    const int per_layer = 2 * kv.heads * c.vecs;
    for (int i = blockIdx.y * kCompactThreads + tid; i < c.layers * per_layer; i += gridDim.y * kCompactThreads) {
        const int layer = i / per_layer, in = i - layer * per_layer;
        const int which = in / (kv.heads * c.vecs), hv = in - which * kv.heads * c.vecs;
        const int h = hv / c.vecs, vec = hv - h * c.vecs;
        T* p = static_cast<T*>(which ? kv.v : kv.k) + layer * c.layer_stride +
               static_cast<int64_t>(h) * kv.block_size() * kv.dim + vec * c.vec_elems;
        for (int m = 0; m < n; ++m)
            *reinterpret_cast<uint4*>(p + s_dst[m]) = *reinterpret_cast<const uint4*>(p + s_src[m]);
    }
}

}  // namespace specv
