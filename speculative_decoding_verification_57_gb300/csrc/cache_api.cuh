// cache_api.cuh -- C ABI of the paged KV cache: argument checks and launches
// of append, tree attention and compaction.  Included behind specv.cu, whose
// handle and error handling it uses.
#pragma once
#include "attention_plan.cuh"
#include "cache_append.cuh"
#include "cache_compact.cuh"

namespace {

using AppendKernel = void (*)(AppendArgs);

template <typename T, int THREADS>
AppendKernel append_kernel_of(int mode) {
    return mode == kApart        ? cache_append_kernel<T, kApart, THREADS>
           : mode == kNeighbours ? cache_append_kernel<T, kNeighbours, THREADS>
                                 : cache_append_kernel<T, kValues, THREADS>;
}

AppendKernel append_kernel(specv_dtype dt, int mode, bool many) {
    using B = __nv_bfloat16;
    if (dt == SPECV_BF16) return many ? append_kernel_of<B, kAppendMany>(mode) : append_kernel_of<B, kAppendFew>(mode);
    return many ? append_kernel_of<float, kAppendMany>(mode) : append_kernel_of<float, kAppendFew>(mode);
}

}  // namespace

extern "C" {

specv_status specv_cache_append(specv_handle h, const specv_kv_cache* cache, const void* q, int64_t q_stride,
                                int q_heads, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                const float* inv_freq, int rot_dim, int interleaved, const int32_t* parents,
                                const int32_t* row_counts, int batch, int rows, void* q_out, int32_t* row_status,
                                void* stream) {
    AppendArgs a = {};
    if (!make_view(h, cache, batch, a.kv)) return SPECV_ERR_INVALID_ARGUMENT;
    if (rows < 1 || (parents && rows - 1 > h->max_k)) return SPECV_ERR_INVALID_ARGUMENT;
    if (static_cast<int64_t>(batch) * rows > INT32_MAX) return SPECV_ERR_INVALID_ARGUMENT;
    if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 2 || (rot_dim > 0 && !inv_freq))
        return SPECV_ERR_INVALID_ARGUMENT;
    if (batch == 0) return SPECV_OK;
    if (!rows_ok(cache, k, k_stride) || !rows_ok(cache, v, v_stride)) return SPECV_ERR_INVALID_ARGUMENT;
    if (q && (!rows_ok(cache, q, q_stride) || !q_out || !aligned16(q_out) || q_heads < 1 || q_heads > 65536 ||
              (q_out == q && q_stride != static_cast<int64_t>(q_heads) * cache->head_dim)))
        return SPECV_ERR_INVALID_ARGUMENT;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.inv_freq = inv_freq;
    a.parents = rows > 1 ? parents : nullptr;
    a.row_counts = row_counts;
    a.row_status = row_status;
    a.q_heads = q ? q_heads : 0;
    a.rot = rot_dim;
    a.interleaved = interleaved != 0;
    a.rows = FastDiv(static_cast<uint32_t>(rows));
    const int vec = cache->dtype == SPECV_BF16 ? 8 : 4;
    a.units = FastDiv(static_cast<uint32_t>(cache->head_dim / vec / 2));
    DeviceGuard g(h->device);
    if (!g.ok) return cuda_fail(cudaErrorInvalidDevice, "cudaSetDevice");
    const unsigned grid = static_cast<unsigned>(batch) * static_cast<unsigned>(rows);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool many = grid > static_cast<unsigned>(h->sm_count) * (kAppendResident / kAppendFew);
    // pieces of 16 bytes turn whole, apart or within, where rot_dim fills them
    const int mode = rot_dim % (interleaved ? vec : 2 * vec) ? kValues : interleaved && rot_dim ? kNeighbours : kApart;
    const AppendKernel kernel = append_kernel(cache->dtype, mode, many);
    kernel<<<grid, many ? kAppendMany : kAppendFew, 0, s>>>(a);
    return launched(h, "cache_append launch");
}

int64_t specv_tree_attention_workspace(specv_handle h, specv_dtype dtype, int kv_heads, int head_dim, int q_heads,
                                       int batch, int rows) {
    if (!h || (dtype != SPECV_F32 && dtype != SPECV_BF16) || kv_heads < 1 || head_dim < 16 || head_dim > 256 ||
        head_dim % 16 || q_heads < 1 || q_heads > 65536 || q_heads % kv_heads || batch < 1 ||
        batch > h->max_batch || rows < 1 || rows - 1 > h->max_k)
        return 0;
    const AttnPlan<AttnArgs>& p = attn_plan<AttnArgs>(dtype, head_dim, rows * (q_heads / kv_heads));
    return attn_work_bytes(h->sm_count * p.ctas, p.tm, p.dp);
}

specv_status specv_tree_attention(specv_handle h, const specv_kv_cache* cache, const void* q, int64_t q_stride,
                                  int q_heads, const int32_t* parents, int batch, int rows, float scale, void* out,
                                  float* lse, int32_t* row_status, void* workspace, int64_t workspace_bytes,
                                  void* stream) {
    AttnArgs a = {};
    if (!make_view(h, cache, batch, a.kv)) return SPECV_ERR_INVALID_ARGUMENT;
    if (rows < 1 || rows - 1 > h->max_k || q_heads < 1 || q_heads > 65536 || q_heads % cache->kv_heads ||
        !std::isfinite(scale) || !std::isfinite(attn_scale(scale)))
        return SPECV_ERR_INVALID_ARGUMENT;
    if (batch == 0) return SPECV_OK;
    // (a segment's end writes its rows of out while others still read their queries)
    if (!rows_ok(cache, q, q_stride) || !out || !aligned16(out) || out == q) return SPECV_ERR_INVALID_ARGUMENT;
    const int group = q_heads / cache->kv_heads;
    const AttnPlan<AttnArgs>& p = attn_plan<AttnArgs>(cache->dtype, cache->head_dim, rows * group);
    const int ctas = h->sm_count * p.ctas;
    if (!workspace || workspace_bytes < attn_work_bytes(ctas, p.tm, p.dp) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255))
        return SPECV_ERR_INVALID_ARGUMENT;
    a.q = q;
    a.q_stride = q_stride;
    a.parents = rows > 1 ? parents : nullptr;
    a.out = out;
    a.lse = lse;
    a.row_status = row_status;
    a.workspace = static_cast<unsigned char*>(workspace);
    a.group = FastDiv(static_cast<uint32_t>(group));
    a.filled = FastDiv(static_cast<uint32_t>(rows * group < p.tm ? rows * group : p.tm));
    a.q_heads = q_heads;
    a.rows = rows;
    a.batch = batch;
    a.row_tiles = (rows * group + p.tm - 1) / p.tm;
    a.scale = scale;
    a.withhold = -1;
    a.polls = 1u << 30;
    if (p.tc && h->test_withhold >= 0) {  // the test hook arms one launch
        a.withhold = h->test_withhold;
        a.polls = h->test_polls;
        h->test_withhold = -1;
    }
    DeviceGuard g(h->device);
    if (!g.ok) return cuda_fail(cudaErrorInvalidDevice, "cudaSetDevice");
    const cudaError_t e = p.launch(a, ctas, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tree_attention launch");
    h->launches.fetch_add(2, std::memory_order_relaxed);
    return SPECV_OK;
}

specv_status specv_cache_compact(specv_handle h, const specv_kv_cache* cache, int layers, int64_t layer_stride,
                                 const int32_t* path, const int32_t* num_accepted, int batch, int M,
                                 int32_t* row_status, void* stream) {
    CompactArgs c = {};
    if (!make_view(h, cache, batch, c.kv)) return SPECV_ERR_INVALID_ARGUMENT;
    const int vec = cache->dtype == SPECV_BF16 ? 8 : 4;
    if (M < 1 || M > h->max_k || layers < 1 || layers > 65536 || layer_stride < 0 || layer_stride % vec)
        return SPECV_ERR_INVALID_ARGUMENT;
    // (layers overlap unless the pools or the blocks of one lie apart; either order of the two strides is fine)
    if (layers > 1 && layer_stride < static_cast<int64_t>(cache->kv_heads) * cache->block_size * cache->head_dim)
        return SPECV_ERR_INVALID_ARGUMENT;
    if (layer_stride > INT64_MAX / 16 / layers) return SPECV_ERR_INVALID_ARGUMENT;
    if (batch == 0) return SPECV_OK;
    if (!path || !num_accepted) return SPECV_ERR_INVALID_ARGUMENT;
    c.path = path;
    c.num_accepted = num_accepted;
    c.row_status = row_status;
    c.layer_stride = layer_stride;
    c.M = M;
    c.layers = layers;
    c.vec_elems = vec;
    DeviceGuard g(h->device);
    if (!g.ok) return cuda_fail(cudaErrorInvalidDevice, "cudaSetDevice");
    const int64_t per_head = cache->head_dim / vec, per_layer = 2 * cache->kv_heads * per_head;
    const int64_t pieces = layers * per_layer;
    if (pieces > INT32_MAX / 2) return SPECV_ERR_INVALID_ARGUMENT;
    c.per_head = FastDiv(static_cast<uint32_t>(per_head));
    c.per_cache = FastDiv(static_cast<uint32_t>(per_layer / 2));
    c.per_layer = FastDiv(static_cast<uint32_t>(per_layer));
    const int64_t want = (pieces + kCompactThreads - 1) / kCompactThreads;
    const dim3 grid(static_cast<unsigned>(batch), static_cast<unsigned>(want < 1 ? 1 : want > kCompactCtas ? kCompactCtas : want), 1);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cache->dtype == SPECV_BF16)
        cache_compact_kernel<__nv_bfloat16><<<grid, kCompactThreads, 0, s>>>(c);
    else
        cache_compact_kernel<float><<<grid, kCompactThreads, 0, s>>>(c);
    return launched(h, "cache_compact launch");
}

}  // extern "C"
