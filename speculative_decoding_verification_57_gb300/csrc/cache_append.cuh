// cache_append.cuh -- keys and values of a pass into the paged cache, queries
// and keys turned by their rotary positions on the way.
//
// A token is a CTA: its position's angles are formed once in shared memory
// and serve every head.  Angles are formed in float64 (position * inv_freq
// passes 2^24 for far positions, where fp32 would lose the fraction of a
// turn), brought into [-pi, pi] there, and the sine and cosine are taken in
// fp32.
#pragma once
#include "kv_cache.cuh"

namespace specv {

constexpr int kAppendThreads = 256;

struct AppendArgs {
    KvView kv;
    const void *q, *k, *v;
    void* q_out;
    int64_t q_stride, k_stride, v_stride;
    const float* inv_freq;
    const int32_t* parents;
    const int32_t* row_counts;
    int32_t* row_status;
    int q_heads, rot, interleaved;
    int rows;
};

// cos and sin of the angle pos * f.
__device__ __forceinline__ float2 append_turn(int pos, float f) {
    const double a = static_cast<double>(pos) * static_cast<double>(f);
    const double two_pi = 6.283185307179586476925286766559;
    const double turns = rint(a * 0.15915494309189533576888376337251);
    float s, c;
    sincosf(static_cast<float>(fma(-turns, two_pi, a)), &s, &c);
    return make_float2(c, s);
}

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendArgs a) {
    __shared__ float2 turn[128];
    __shared__ int s_status;
    const int b = blockIdx.x / a.rows, r = blockIdx.x % a.rows;
    const int tid = threadIdx.x;
    const KvView& kv = a.kv;
    const int len = kv.lens[b];
    const int count = a.row_counts ? a.row_counts[b] : (len == 0 ? 0 : a.rows);
    int status = 0;
    if (count < 0 || count > a.rows || len < 0 || (count > 0 && (len < count || !kv.fits(len)))) status = KV_LENGTH;
    const int base = len - count;
    // every token of a sequence looks at all its blocks: a refused sequence writes nothing
    if (tid == 0) s_status = 0;
    __syncthreads();
    int depth = r;
    if (status == 0 && count > 0) {
        if (a.parents && tid < 32) {
            uint32_t anc;
            int d;
            const bool ok = warp_tree(a.parents + static_cast<int64_t>(b) * (a.rows - 1), count, tid, anc, d);
            if (!ok && tid == 0) atomicOr(&s_status, KV_PARENT);
            if (tid == r) turn[0].x = __int_as_float(d);
        }
        const int first = kv.block.div(base), last = kv.block.div(len - 1);
        for (int i = first + tid; i <= last; i += kAppendThreads)
            if (!kv.valid(kv.tables[static_cast<int64_t>(b) * kv.max_blocks + i])) atomicOr(&s_status, KV_BLOCK);
        __syncthreads();
        status = s_status;
        if (a.parents) depth = __float_as_int(turn[0].x);
        __syncthreads();
    }
    if (r == 0 && tid == 0 && a.row_status) a.row_status[b] = status;
    const int64_t token = static_cast<int64_t>(b) * a.rows + r;
    const T* q = static_cast<const T*>(a.q) + token * a.q_stride;
    T* q_out = static_cast<T*>(a.q_out) + token * a.q_heads * kv.dim;
    if (status != 0 || r >= count) {
        if (a.q)
            for (int i = tid; i < a.q_heads * kv.dim; i += kAppendThreads) q_out[i] = KvType<T>::store(0.0f);
        return;
    }
    const int half = a.rot / 2;
    for (int j = tid; j < half; j += kAppendThreads) turn[j] = append_turn(base + depth, a.inv_freq[j]);
    __syncthreads();
    const int slot = base + r;
    const int lb = kv.block.div(slot), in = slot - lb * kv.block_size();
    const int blk = kv.tables[static_cast<int64_t>(b) * kv.max_blocks + lb];
    const T* k = static_cast<const T*>(a.k) + token * a.k_stride;
    const T* v = static_cast<const T*>(a.v) + token * a.v_stride;
    const int q_n = a.q ? a.q_heads : 0;
    const int pairs = kv.dim / 2;  // of a head: half rotated pairs, then the rest by twos
    for (int i = tid; i < (q_n + kv.heads) * pairs; i += kAppendThreads) {
        int h = i / pairs, j = i - h * pairs;
        const bool is_q = h < q_n;
        if (!is_q) h -= q_n;
        const T* x = is_q ? q + h * kv.dim : k + h * kv.dim;
        T* y = is_q ? q_out + h * kv.dim : static_cast<T*>(kv.k) + kv.at(blk, h, in);
        const int i0 = j >= half || a.interleaved ? 2 * j : j;
        const int i1 = j >= half || a.interleaved ? 2 * j + 1 : j + half;
        if (j >= half) {
            y[i0] = x[i0];
            y[i1] = x[i1];
        } else {
            const float x0 = KvType<T>::load(x[i0]), x1 = KvType<T>::load(x[i1]);
            const float2 cs = turn[j];
            y[i0] = KvType<T>::store(x0 * cs.x - x1 * cs.y);
            y[i1] = KvType<T>::store(x0 * cs.y + x1 * cs.x);
        }
    }
    for (int i = tid; i < kv.heads * kv.dim; i += kAppendThreads) {
        const int h = i / kv.dim, d = i - h * kv.dim;
        static_cast<T*>(kv.v)[kv.at(blk, h, in) + d] = v[i];
    }
}

}  // namespace specv
