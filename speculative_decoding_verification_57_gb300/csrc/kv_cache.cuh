// kv_cache.cuh -- what the kernels on the paged KV cache share: the cache as
// a kernel sees it, the checks of a sequence, and the tree of a pass's rows
// ("LLM Inference & Speculative Decoding: From Roofline Physics to Lossless
// Acceleration", s.1 PagedKVCacheManager, s.3 the ancestor mask and depths).
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

namespace specv {

enum : int { KV_TIMEOUT = 64, KV_PARENT = 512, KV_LENGTH = 2048, KV_BLOCK = 4096, KV_PATH = 8192, KV_ACCEPTED = 128 };

// Quotients n / d of 0 <= n < 2^31 by one multiplication: with p = 31 +
// ceil(log2 d), m = ceil(2^p / d) is below 2^32 and off by less than d, so
// that n * m / 2^p is off by less than n / 2^p * 1 <= 2^-ceil(log2 d) <= 1/d.
struct FastDiv {
    uint32_t mul = 0, shift = 0, d = 1;  // mul 0: d = 1
    FastDiv() = default;
    explicit FastDiv(uint32_t div) : d(div) {
        if (div == 1) return;
        uint32_t lg = 0;
        while ((1ull << lg) < div) ++lg;
        mul = static_cast<uint32_t>(((1ull << (31 + lg)) + div - 1) / div);
        shift = lg - 1;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return mul ? __umulhi(n, mul) >> shift : n; }
};

struct KvView {
    void *k, *v;
    const int32_t* tables;  // [B, max_blocks]
    const int32_t* lens;    // [B]
    int64_t block_stride;   // elements
    int blocks, max_blocks;
    int heads, dim;
    FastDiv block;  // by block_size

    __device__ __forceinline__ int block_size() const { return static_cast<int>(block.d); }
    // offset, in elements, of position `slot` (inside its block) of head h
    __device__ __forceinline__ int64_t at(int blk, int h, int slot) const {
        return blk * block_stride + (static_cast<int64_t>(h) * block_size() + slot) * dim;
    }
    // whether n positions fit the table (and a tile beyond them an int)
    __device__ __forceinline__ bool fits(int n) const {
        return n <= static_cast<int64_t>(max_blocks) * block_size() && n <= INT32_MAX - 512;
    }
    __device__ __forceinline__ bool valid(int blk) const { return blk >= 0 && blk < blocks; }
};

// The tree of one sequence's rows, by one converged warp; lane r holds row r
// (row 0 the root, row 1 + i node i) and, as `parent`, parents[r - 1].  anc:
// bit j set if row j is row r or above it.  Pointers are doubled, so five
// steps reach the root of any tree of 32 rows.  Returns false (in every lane)
// if a parent is outside [-1, i); lanes past `rows` hold nothing.
__device__ __forceinline__ bool warp_tree_of(int parent, int rows, int lane, uint32_t& anc, int& depth) {
    const bool node = lane > 0 && lane < rows;
    const bool ok = !node || (parent >= -1 && parent < lane - 1);
    int up = node && ok ? parent + 1 : 0;  // the row above; the root's is itself
    const bool all_ok = __all_sync(0xffffffffu, ok);
    anc = lane < rows ? (1u << lane) | (1u << up) : 0;
#pragma unroll
    for (int step = 0; step < 5; ++step) {
        anc |= __shfl_sync(0xffffffffu, anc, up);
        up = __shfl_sync(0xffffffffu, up, up);
    }
    if (lane >= rows) anc = 0;
    depth = __popc(anc) - 1;
    return all_ok;
}

// The same from the sequence's parents in memory (NULL: a chain).
__device__ __forceinline__ bool warp_tree(const int32_t* parents, int rows, int lane, uint32_t& anc, int& depth) {
    const int parent = parents && lane > 0 && lane < rows ? parents[lane - 1] : lane - 2;
    return warp_tree_of(parent, rows, lane, anc, depth);
}

template <typename T>
struct KvType;
template <>
struct KvType<float> {
    static constexpr int kVec = 4;  // elements in 16 bytes
    static __device__ __forceinline__ float load(float x) { return x; }
    static __device__ __forceinline__ float store(float x) { return x; }
};
template <>
struct KvType<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float load(__nv_bfloat16 x) { return __bfloat162float(x); }
    // to nearest: the one rounding of a value that leaves in 16 bits
    static __device__ __forceinline__ __nv_bfloat16 store(float x) { return __float2bfloat16_rn(x); }
};

__device__ __forceinline__ uint32_t kv_pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 16 bytes of elements.
template <typename T>
struct alignas(16) KvVec {
    T x[KvType<T>::kVec];
};

}  // namespace specv
