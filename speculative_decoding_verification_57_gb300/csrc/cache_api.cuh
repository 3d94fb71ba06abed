// cache_api.cuh -- C ABI of the paged KV cache: argument checks and launches
// of append, tree attention and compaction.  Included behind specv.cu, whose
// handle and error handling it uses.
#pragma once
#include "cache_append.cuh"
#include "cache_compact.cuh"
#include "tree_attention.cuh"
#include "tree_attention_tc.cuh"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The cache of a call as the kernels see it; false if a size, pointer or
// alignment is outside what specv_kv_cache allows.
bool make_view(const specv_ctx* h, const specv_kv_cache* c, int batch, KvView& view) {
    if (!h || !c || batch < 0 || batch > h->max_batch) return false;
    if (c->dtype != SPECV_F32 && c->dtype != SPECV_BF16) return false;
    if (c->kv_heads < 1 || c->kv_heads > 65536 || c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
        return false;
    if (c->block_size < 1 || c->block_size > 65536 || c->max_blocks < 0 || c->blocks < 0 || c->blocks > INT32_MAX)
        return false;
    const int64_t inner = static_cast<int64_t>(c->kv_heads) * c->block_size * c->head_dim;
    const int64_t vec = c->dtype == SPECV_BF16 ? 8 : 4;
    if (c->block_stride < inner || c->block_stride % vec) return false;
    if (c->block_stride > INT64_MAX / 8 / (c->blocks > 0 ? c->blocks : 1)) return false;
    if (batch > 0 && (!c->seq_lens || (c->max_blocks > 0 && !c->block_tables) || (c->blocks > 0 && (!c->k || !c->v))))
        return false;
    if (!aligned16(c->k) || !aligned16(c->v)) return false;
    view.k = c->k;
    view.v = c->v;
    view.tables = c->block_tables;
    view.lens = c->seq_lens;
    view.block_stride = c->block_stride;
    view.blocks = static_cast<int>(c->blocks);
    view.max_blocks = c->max_blocks;
    view.heads = c->kv_heads;
    view.dim = c->head_dim;
    view.block = FastDiv(static_cast<uint32_t>(c->block_size));
    return true;
}

// A tensor of rows [.., heads, head_dim]: its pointer and row stride.
bool rows_ok(const specv_kv_cache* c, const void* p, int64_t stride) {
    const int64_t vec = c->dtype == SPECV_BF16 ? 8 : 4;
    return p && aligned16(p) && stride >= 0 && stride % vec == 0;
}

// Launch errors of the calls below.
specv_status launched(specv_ctx* h, const char* what) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, what);
    h->launches.fetch_add(1, std::memory_order_relaxed);
    return SPECV_OK;
}

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

// Tree attention of one shape: its kernel and, behind it, the join.  The CTAs
// of both may be placed while the kernel before still runs (they wait for its
// end on the device), so that launches overlap what runs before them.
template <typename... Params>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t stream,
                         const Params&... params) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, params...);
}

template <typename S>
cudaError_t launch_join(const AttnArgs& a, int ctas, cudaStream_t stream) {
    // Many segments, at most two or three pieces each, if there are half as many as CTAs; sixteen columns a thread pay
    // for row tiles of 256 (16 trees of 32 rows with 64 heads: 113 us for 118), and cost chains of 6 rows 83 us for 80
    const bool few = static_cast<int64_t>(a.batch) * a.kv.heads * a.row_tiles < ctas / 2;
    constexpr int kCols = S::TM == 256 ? 4 : 1;
    const int threads = static_cast<int>(a.filled.d) * (a.kv.dim / (few ? 4 : 4 * kCols));  // of a segment
    const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>((threads + kJoinThreads - 1) / kJoinThreads));
    return launch_early(few ? tree_attention_join<S, 8, 1> : tree_attention_join<S, 2, kCols>, grid, kJoinThreads, 0, stream,
                        a, ctas);
}

// Lets a kernel have `bytes` of dynamic shared memory; once a device (a bit
// of `done` each) is enough.
cudaError_t allow_smem(std::atomic<uint64_t>& done, const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <typename S>
cudaError_t launch_attention(const AttnArgs& a, int ctas, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(tree_attention_kernel<S>), S::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_early(tree_attention_kernel<S>, dim3(static_cast<unsigned>(ctas)), S::kThreads, S::kSmem, stream, a);
    return e != cudaSuccess ? e : launch_join<S>(a, ctas, stream);
}

// Boxes for the cache's blocks, if they fill tiles of 128 rows evenly; false:
// they do not, or the pool is outside what a tensor map can say.
bool make_maps(const AttnArgs& a, TcMaps& maps) {
    const KvView& kv = a.kv;
    const int bs = static_cast<int>(kv.block.d);
    if (bs % 8 || (128 % bs && bs % 128) || kv.blocks < 1 || kv.block_stride >= (1ll << 38)) return false;
    static const auto encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                             CUtensorMapFloatOOBfill)>(f);
    }();
    if (!encode) return false;
    maps.rows = bs < 128 ? bs : 128;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.dim), static_cast<cuuint64_t>(bs),
                                static_cast<cuuint64_t>(kv.heads), static_cast<cuuint64_t>(kv.blocks)};
    const cuuint64_t strides[3] = {dims[0] * 2, dims[0] * dims[1] * 2, static_cast<cuuint64_t>(kv.block_stride) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(maps.rows), 1, 1}, ones[4] = {1, 1, 1, 1};
    for (int i = 0; i < 2; ++i)
        if (encode(i ? &maps.v : &maps.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, i ? kv.v : kv.k, dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    // the queries, a row tile a box and panel, where groups of heads fill row tiles
    const int group = static_cast<int>(a.group.d);
    maps.q_rows = 0;
    if (128 % group == 0 && a.q_stride > 0 && a.q_stride * a.rows < (1ll << 38)) {
        const cuuint64_t q_dims[4] = {dims[0], static_cast<cuuint64_t>(a.q_heads), static_cast<cuuint64_t>(a.rows),
                                      static_cast<cuuint64_t>(a.batch)};
        const cuuint64_t q_strides[3] = {dims[0] * 2, static_cast<cuuint64_t>(a.q_stride) * 2,
                                         static_cast<cuuint64_t>(a.q_stride) * a.rows * 2};
        const cuuint32_t q_box[4] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(128 / group), 1};
        if (encode(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.q), q_dims, q_strides, q_box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
            maps.q_rows = 128 / group;
    }
    return true;
}

template <typename S>
cudaError_t launch_tc(const AttnArgs& a, const TcMaps& maps, int ctas, cudaStream_t stream) {
    constexpr int kBytes = sizeof(TcShared<S>);
    static_assert(kBytes <= 227 * 1024, "a CTA's shared memory");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(tree_attention_tc_kernel<S>), kBytes);
    if (e != cudaSuccess) return e;
    e = launch_early(tree_attention_tc_kernel<S>, dim3(static_cast<unsigned>(ctas)), S::kThreads, kBytes, stream, a, maps);
    return e != cudaSuccess ? e : launch_join<S>(a, ctas, stream);
}

template <int DP, bool WIDE>
cudaError_t launch_attention_tc(const AttnArgs& a, int ctas, cudaStream_t stream) {
    TcMaps maps = {};
    if (make_maps(a, maps)) return launch_tc<TcShape<DP, WIDE, true>>(a, maps, ctas, stream);
    return launch_tc<TcShape<DP, WIDE, false>>(a, maps, ctas, stream);
}

struct AttnPlan {
    int dp, tm, ctas;  // padded head_dim, rows of a tile, CTAs an SM
    bool tc;           // the tcgen05 kernel
    cudaError_t (*launch)(const AttnArgs&, int, cudaStream_t);
};

template <typename S>
constexpr AttnPlan plan_of() {
    return AttnPlan{S::DP, S::TM, S::kCtas, false, launch_attention<S>};
}

template <int DP, bool WIDE>
constexpr AttnPlan plan_of_tc() {
    return AttnPlan{DP, TcShape<DP, WIDE, true>::TM, 1, true, launch_attention_tc<DP, WIDE>};
}

// bf16 rows up to head_dim 128 and more than 16 rows a kv head (rows * group)
// go to the tcgen05 kernel, whose row tile of 128 costs the tensor cores less
// time than its positions cost the memory; up to 16 the other's pipeline is
// shorter.  Single rows, 32/8 heads of 128, this kernel | the tcgen05 one, us:
//   sequences   500 positions   2000          20,000        131,072
//   1           9.0 | 11.2      14.5 | 14.3   28.9 | 27.6   99 | 92
//   4           10.4 | 12.6     16.7 | 19.4   54.0 | 52.4   285 | 264
//   64          32.5 | 44.8     75.1 | 76.0   618 | 577
// (4 rows, 16 a kv head, within 3% of these); 16 heads of 64, 128 single rows
// over 1000 positions 89 | 150, 16 rows for 64 over 2000 82 | 108, for 4 over
// 20,000 56 | 60.  So long contexts of heads of 128 would be 3 to 8% faster
// there; but lengths are device memory, and the rule does not look at them.  Of
// 20 rows a kv head, 64 sequences over 300 positions take 42.3 us on this
// kernel (with a row tile of 32) and 36.6 there, 1 over 2000 13.7 and 14.6.  In
// each, the narrowest row tile that holds the rows, or the widest: a tile's
// keys and values are read once for all of its rows.
constexpr int kTcLeast = 17;

const AttnPlan& attn_plan(specv_dtype dt, int dim, int m) {
    using B = __nv_bfloat16;
    using F = float;
    static constexpr AttnPlan f32[3][3] = {
        {plan_of<AttnShape<F, 64, 1, 1>>(), plan_of<AttnShape<F, 64, 1, 2>>(), plan_of<AttnShape<F, 64, 2, 2>>()},
        {plan_of<AttnShape<F, 128, 1, 1>>(), plan_of<AttnShape<F, 128, 1, 2>>(), plan_of<AttnShape<F, 128, 2, 2>>()},
        {plan_of<AttnShape<F, 256, 1, 1>>(), plan_of<AttnShape<F, 256, 1, 2>>(), plan_of<AttnShape<F, 256, 1, 2>>()}};
    static constexpr AttnPlan few[2] = {plan_of<AttnShape<B, 64, 1, 1>>(), plan_of<AttnShape<B, 128, 1, 1>>()};
    static constexpr AttnPlan many[2][2] = {{plan_of_tc<64, false>(), plan_of_tc<64, true>()},
                                            {plan_of_tc<128, false>(), plan_of_tc<128, true>()}};
    static constexpr AttnPlan big[2] = {plan_of<AttnShape<B, 256, 1, 1>>(), plan_of<AttnShape<B, 256, 1, 2>>()};
    const int d = dim <= 64 ? 0 : dim <= 128 ? 1 : 2;
    if (dt == SPECV_F32) return f32[d][m <= 16 ? 0 : m <= 32 ? 1 : 2];
    if (d == 2) return big[m <= 16 ? 0 : 1];
    return m < kTcLeast ? few[d] : many[d][m <= 128 ? 0 : 1];
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
    const AttnPlan& p = attn_plan(dtype, head_dim, rows * (q_heads / kv_heads));
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
    const AttnPlan& p = attn_plan(cache->dtype, cache->head_dim, rows * group);
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
