// tree_attention.cuh -- attention of a pass's rows (a chain or a tree of
// drafted tokens) over the paged cache.
//
// Row r of sequence b sees the positions before the pass's rows and, of
// these, itself and its ancestors.  o = sum_j p_j v_j / sum_j p_j with
// p_j = exp(scale q.k_j - m), m the running maximum of the scores seen so far.
#pragma once
#include "kv_cache.cuh"

namespace specv {

constexpr int kAttnThreads = 128;

struct AttnArgs {
    KvView kv;
    const void* q;
    int64_t q_stride;
    const int32_t* parents;
    void* out;
    float* lse;
    int32_t* row_status;
    int q_heads, group, rows;
    float scale;
};

template <typename T>
__global__ void __launch_bounds__(kAttnThreads) tree_attention_kernel(const AttnArgs a) {
    __shared__ float s_q[256], s_p[kAttnThreads], s_red[4];
    __shared__ int s_blk[kAttnThreads], s_status;
    __shared__ uint32_t s_anc;
    const int h = blockIdx.x, r = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const KvView& kv = a.kv;
    const int dim = kv.dim, kvh = h / a.group;
    const int len = kv.lens[b];
    if (tid < 32) {
        uint32_t anc;
        int depth;
        const bool ok = warp_tree(a.parents ? a.parents + static_cast<int64_t>(b) * (a.rows - 1) : nullptr, a.rows,
                                  tid, anc, depth);
        if (tid == r) s_anc = anc;
        if (tid == 0) {
            s_status = ok || len == 0 ? 0 : KV_PARENT;
            if (len < 0 || (len > 0 && (len < a.rows || !kv.fits(len)))) s_status |= KV_LENGTH;
        }
    }
    const int64_t token = static_cast<int64_t>(b) * a.rows + r;
    const T* q = static_cast<const T*>(a.q) + token * a.q_stride + h * dim;
    T* out = static_cast<T*>(a.out) + (token * a.q_heads + h) * dim;
    for (int d = tid; d < dim; d += kAttnThreads) s_q[d] = KvType<T>::load(q[d]);
    __syncthreads();
    const uint32_t anc = s_anc;
    const int base = len - a.rows;
    float m = -INFINITY, sum = 0.0f, acc[2] = {0.0f, 0.0f};
    const bool go = s_status == 0 && len > 0;
    __syncthreads();
    for (int t0 = 0; go && t0 < len; t0 += kAttnThreads) {
        const int t = t0 + tid;
        float s = -INFINITY;
        int blk = -1;
        if (t < len) {
            const int lb = kv.block.div(t);
            blk = kv.tables[static_cast<int64_t>(b) * kv.max_blocks + lb];
            if (!kv.valid(blk)) {
                s_status = KV_BLOCK;
                blk = -1;
            } else if (t < base || (anc >> (t - base) & 1)) {
                const T* k = static_cast<const T*>(kv.k) + kv.at(blk, kvh, t - lb * kv.block_size());
                s = 0.0f;
                for (int d = 0; d < dim; ++d) s = fmaf(s_q[d], KvType<T>::load(k[d]), s);
                s *= a.scale;
            } else {
                blk = -1;
            }
        }
        float top = s;
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        if ((tid & 31) == 0) s_red[tid >> 5] = top;
        __syncthreads();
        const float m_new = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
        const float m_use = m_new == -INFINITY ? 0.0f : m_new;
        s_p[tid] = blk >= 0 ? expf(s - m_use) : 0.0f;
        s_blk[tid] = blk;
        __syncthreads();
        const float keep = expf(m - m_use);
        m = m_new;
        sum *= keep;
        acc[0] *= keep;
        acc[1] *= keep;
        const int n = min(kAttnThreads, len - t0);
        for (int i = 0; i < n; ++i) {
            if (s_blk[i] < 0) continue;
            sum += s_p[i];
            const int lb = kv.block.div(t0 + i);
            const T* v = static_cast<const T*>(kv.v) + kv.at(s_blk[i], kvh, t0 + i - lb * kv.block_size());
            if (tid < dim) acc[0] = fmaf(s_p[i], KvType<T>::load(v[tid]), acc[0]);
            if (tid + kAttnThreads < dim) acc[1] = fmaf(s_p[i], KvType<T>::load(v[tid + kAttnThreads]), acc[1]);
        }
        __syncthreads();
    }
    const bool fine = go && s_status == 0;
    if (h == 0 && r == 0 && tid == 0 && a.row_status) a.row_status[b] = s_status;
    for (int i = 0; i < 2; ++i)
        if (tid + i * kAttnThreads < dim) out[tid + i * kAttnThreads] = KvType<T>::store(fine ? acc[i] / sum : 0.0f);
    if (tid == 0 && a.lse) a.lse[token * a.q_heads + h] = fine ? m + logf(sum) : -INFINITY;
}

}  // namespace specv
