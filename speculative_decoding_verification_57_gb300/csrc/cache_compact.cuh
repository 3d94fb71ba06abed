// cache_compact.cuh -- the kept path of a verified tree moved together in the
// paged cache, keys and values of every layer in one launch.
//
// Node path[i] goes to the place of node i.  A path is strictly increasing,
// so path[i] >= i: no place is written before it was read if the moves run in
// order of i, and a thread that owns the same 16 bytes of every node can run
// them without a barrier, four loads ahead of their stores at a time (a
// place stored to is never one that a later move reads).  Nodes that are in
// place already are left out.
//
// Measured (GB300, graph replays over sets of inputs of more than twice the
// L2): 32 layers of 64 sequences, up to 4 nodes of 8 heads of 128 in bf16 each,
// 7.5 us, 68% of 6691 GB/s for 34 MB (5.8 with inputs in the L2); one layer of 8
// sequences 2.0 us.  Bound by the chain length, table, node, which at most
// twelve CTAs a sequence go through (64: 7.5 us too, 6.2 in the L2).
#pragma once
#include "kv_cache.cuh"

namespace specv {

constexpr int kCompactThreads = 256;
constexpr int kCompactCtas = 12;  // of a sequence at most
constexpr int kCompactMoves = 4;  // of a thread, in flight

struct CompactArgs {
    KvView kv;
    const int32_t* path;          // [B, M]
    const int32_t* num_accepted;  // [B]
    int32_t* row_status;
    int64_t layer_stride;  // elements
    int M, layers;
    FastDiv per_layer;  // pieces of 16 bytes of a node in a layer, keys and values
    FastDiv per_cache;  // ... in keys or values
    FastDiv per_head;   // ... in a head
    int vec_elems;
};

template <typename T>
__global__ void __launch_bounds__(kCompactThreads, 6) cache_compact_kernel(const CompactArgs c) {
    __shared__ int64_t s_src[32], s_dst[32];
    __shared__ int s_status, s_moves;
    const int b = blockIdx.x, tid = threadIdx.x;
    const KvView& kv = c.kv;
    if (tid < 32) {
        const int len = kv.lens[b], n = c.num_accepted[b];
        const int seen = tid < c.M ? c.path[static_cast<int64_t>(b) * c.M + tid] : -1;
        int status = 0;
        if (len != 0) {
            if (n < 0 || n > c.M) status |= KV_ACCEPTED;
            if (len < c.M || !kv.fits(len)) status |= KV_LENGTH;
        }
        const bool kept = status == 0 && len != 0 && tid < n;
        const int before = __shfl_up_sync(0xffffffffu, seen, 1);
        const bool path_ok = !kept || (seen >= 0 && seen < c.M && (tid == 0 || seen > before));
        if (!__all_sync(0xffffffffu, path_ok)) status |= KV_PATH;
        bool block_ok = true;
        int64_t from = 0, to = 0;
        if (status == 0 && kept) {
            const int32_t* table = kv.tables + static_cast<int64_t>(b) * kv.max_blocks;
            const int src = len - c.M + seen, dst = len - c.M + tid;
            const int ls = kv.block.div(src), ld = kv.block.div(dst);
            const int bs = table[ls], bd = table[ld];
            block_ok = kv.valid(bs) && kv.valid(bd);
            from = kv.at(bs, 0, src - ls * kv.block_size());
            to = kv.at(bd, 0, dst - ld * kv.block_size());
        }
        if (!__all_sync(0xffffffffu, block_ok)) status |= KV_BLOCK;
        const uint32_t moves = __ballot_sync(0xffffffffu, status == 0 && kept && seen != tid);
        if (moves >> tid & 1) {
            const int at = __popc(moves & ((1u << tid) - 1));
            s_src[at] = from;
            s_dst[at] = to;
        }
        if (tid == 0) {
            s_status = status;
            s_moves = __popc(moves);
            if (blockIdx.y == 0 && c.row_status) c.row_status[b] = status;
        }
    }
    __syncthreads();
    if (s_status != 0) return;
    const int n = s_moves;
    const uint32_t all = static_cast<uint32_t>(c.layers) * c.per_layer.d;
    for (uint32_t i = blockIdx.y * kCompactThreads + tid; i < all; i += gridDim.y * kCompactThreads) {
        const uint32_t layer = c.per_layer.div(i), in = i - layer * c.per_layer.d;
        const uint32_t which = c.per_cache.div(in), hv = in - which * c.per_cache.d;
        const uint32_t h = c.per_head.div(hv), vec = hv - h * c.per_head.d;
        T* p = static_cast<T*>(which ? kv.v : kv.k) + layer * c.layer_stride +
               static_cast<int64_t>(h) * kv.block_size() * kv.dim + vec * c.vec_elems;
        for (int m0 = 0; m0 < n; m0 += kCompactMoves) {
            uint4 x[kCompactMoves];
#pragma unroll
            for (int m = 0; m < kCompactMoves; ++m)
                if (m0 + m < n) x[m] = *reinterpret_cast<const uint4*>(p + s_src[m0 + m]);
#pragma unroll
            for (int m = 0; m < kCompactMoves; ++m)
                if (m0 + m < n) *reinterpret_cast<uint4*>(p + s_dst[m0 + m]) = x[m];
        }
    }
}

}  // namespace specv
