// prefix.cu -- C ABI of attention over a shared prefix.  A translation unit of
// its own, compiled beside library.cu.
#include <cmath>

#include "attention_plan.cuh"
#include "prefix_attention.cuh"

namespace {

constexpr int kOwnUses = 1 << 20;  // of the test hook: uses of the sequences' launch are counted from here

// The launches of a call: its kernels, and what each part needs of the workspace.
struct PrefixPlan {
    const AttnPlan<PartArgs>*prefix, *own;
    int prefix_ctas, own_ctas, prefix_tiles, own_tiles, side;
    int64_t prefix_bytes, own_bytes;
};

PrefixPlan prefix_plan(const specv_ctx* h, specv_dtype dt, int heads, int dim, int group, int batch, int rows) {
    PrefixPlan p;
    const int own = rows * group, all = batch * own;
    // Row tiles of 128 up to eight a kv head, side by side over the same positions, so that they read them from the L2 at
    // about the same time; more rows take tiles of 256, which read the positions half as often (32/8 heads of 128 behind 65536
    // positions, side by side and in tiles of 256: 384 rows 109 and 132 us, 896 207 and 229, 1024 224 and 230, 1152 254 and
    // 267, 1280 263 and 252, 2048 419 and 399; behind 8192, 1024 rows 67 and 69, 1280 65 and 66, 2048 94 and 90)
    const int side = (all + 127) / 128;
    p.prefix = &attn_plan<PartArgs>(dt, dim, all);
    p.side = 1;
    if (p.prefix->tc && side > 1 && side <= 8) {
        p.prefix = &side_plan(dim);
        p.side = side;
    }
    p.own = &attn_plan<PartArgs>(dt, dim, own);
    // ... and beside them the sequences' part goes the same way (16 chains of 6 rows behind 65536 positions 105 us; on twelve
    // warps 110, behind 16384 52 and 57; beside tiles of 256 twelve are as good: 64 chains behind 16384 128 and 126)
    if (p.side > 1 && p.own->tc && own <= 128) p.own = &side_plan(dim);
    p.prefix_ctas = h->sm_count * p.prefix->ctas;
    p.own_ctas = h->sm_count * p.own->ctas;
    p.prefix_tiles = (all + p.prefix->tm - 1) / p.prefix->tm;
    p.own_tiles = (own + p.own->tm - 1) / p.own->tm;
    p.prefix_bytes =
        part_work_bytes(p.prefix_ctas, static_cast<int64_t>(heads) * p.prefix_tiles, p.prefix->tm, p.prefix->dp);
    p.own_bytes = part_work_bytes(p.own_ctas, static_cast<int64_t>(batch) * heads * p.own_tiles, p.own->tm, p.own->dp);
    return p;
}

// Sizes of a call: the rows of a kv head and the threads of the join are counted in 32 bits.
bool prefix_sizes(const specv_ctx* h, int heads, int dim, int q_heads, int batch, int rows) {
    if (rows < 1 || rows - 1 > h->max_k || q_heads < 1 || q_heads > 65536 || q_heads % heads) return false;
    return static_cast<int64_t>(batch) * rows * q_heads * (dim / 4) <= INT32_MAX - kPrefixJoinThreads;
}

template <typename T>
auto prefix_join(bool many) {
    return many ? prefix_join_kernel<T, 4, 2> : prefix_join_kernel<T, 1, 8>;
}

PartView part_view(unsigned char* w, const AttnPlan<PartArgs>& p, int ctas, int row_tiles, int side, int64_t segs) {
    PartView v;
    v.workspace = w;
    v.segs = segs;
    v.ctas = ctas;
    v.tm = p.tm;
    v.row_tiles = row_tiles;
    v.side = side;
    v.dp = p.dp;
    v.tile = FastDiv(static_cast<uint32_t>(p.tm));
    return v;
}

}  // namespace

extern "C" {

int64_t specv_prefix_attention_workspace(specv_handle h, specv_dtype dtype, int kv_heads, int head_dim, int q_heads,
                                         int batch, int rows) {
    if (!h || (dtype != SPECV_F32 && dtype != SPECV_BF16) || kv_heads < 1 || head_dim < 16 || head_dim > 256 ||
        head_dim % 16 || batch < 1 || batch > h->max_batch || !prefix_sizes(h, kv_heads, head_dim, q_heads, batch, rows))
        return 0;
    const PrefixPlan p = prefix_plan(h, dtype, kv_heads, head_dim, q_heads / kv_heads, batch, rows);
    return p.prefix_bytes + p.own_bytes;
}

specv_status specv_prefix_attention(specv_handle h, const specv_kv_cache* cache, const int32_t* prefix_table,
                                    int prefix_blocks, const int32_t* prefix_len, const void* q, int64_t q_stride,
                                    int q_heads, const int32_t* parents, int batch, int rows, float scale, void* out,
                                    float* lse, int32_t* row_status, void* workspace, int64_t workspace_bytes,
                                    void* stream) {
    PartArgs own = {};
    if (!make_view(h, cache, batch, own.kv)) return SPECV_ERR_INVALID_ARGUMENT;
    if (!prefix_sizes(h, cache->kv_heads, cache->head_dim, q_heads, batch, rows) || prefix_blocks < 0 ||
        !std::isfinite(scale) || !std::isfinite(attn_scale(scale)))
        return SPECV_ERR_INVALID_ARGUMENT;
    if (batch == 0) return SPECV_OK;
    if (!rows_ok(cache, q, q_stride) || !out || !aligned16(out) || out == q || !prefix_len ||
        (prefix_blocks > 0 && !prefix_table))
        return SPECV_ERR_INVALID_ARGUMENT;
    const int group = q_heads / cache->kv_heads;
    const PrefixPlan p = prefix_plan(h, cache->dtype, cache->kv_heads, cache->head_dim, group, batch, rows);
    if (!workspace || workspace_bytes < p.prefix_bytes + p.own_bytes || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return SPECV_ERR_INVALID_ARGUMENT;
    const int64_t held = static_cast<int64_t>(prefix_blocks) * cache->block_size;
    own.q = q;
    own.q_stride = q_stride;
    own.parents = rows > 1 ? parents : nullptr;
    own.workspace = static_cast<unsigned char*>(workspace) + p.prefix_bytes;
    own.group = FastDiv(static_cast<uint32_t>(group));
    own.q_heads = q_heads;
    own.rows = own.own = rows;
    own.batch = batch;
    own.row_tiles = p.own_tiles;
    own.side = 1;
    own.scale = scale;
    own.withhold = -1;
    own.polls = 1u << 30;
    own.prefix = prefix_len;
    own.prefix_cap = static_cast<int>(held < INT32_MAX - 512 ? held : INT32_MAX - 512);
    PartArgs all = own;  // the prefix: one sequence with the rows of all
    all.kv.tables = prefix_table;
    all.kv.lens = prefix_len;
    all.kv.max_blocks = prefix_blocks;
    all.parents = nullptr;
    all.workspace = static_cast<unsigned char*>(workspace);
    all.rows = batch * rows;
    all.own = 0;
    all.batch = 1;
    all.row_tiles = p.prefix_tiles;
    all.side = p.side;
    all.prefix = nullptr;
    // the sequences' part before the prefix's where these can run side by side, else behind it
    const bool beside = p.prefix->tc && p.own->tc;
    all.late = beside;
    own.late = !beside;
    if (beside) {
        own.lens = all.lens = cache->seq_lens;
        own.prefix_len = all.prefix_len = prefix_len;
        own.sequences = all.sequences = batch;
        own.own_segs = all.own_segs = cache->kv_heads * p.own_tiles;
        own.prefix_segs = all.prefix_segs = cache->kv_heads * ((batch * rows * group + 127) / 128);
    }
    // the test hook arms one launch: the prefix's, or by numbers from kOwnUses on the sequences'
    PartArgs& armed = h->test_withhold < kOwnUses ? all : own;
    if ((&armed == &all ? p.prefix : p.own)->tc && h->test_withhold >= 0) {
        armed.withhold = h->test_withhold % kOwnUses;
        armed.polls = h->test_polls;
        h->test_withhold = -1;
    }
    PrefixJoinArgs j = {};
    j.prefix = part_view(all.workspace, *p.prefix, p.prefix_ctas, p.prefix_tiles, all.side,
                         static_cast<int64_t>(cache->kv_heads) * p.prefix_tiles);
    j.own = part_view(own.workspace, *p.own, p.own_ctas, p.own_tiles, 1,
                      static_cast<int64_t>(batch) * cache->kv_heads * p.own_tiles);
    j.lens = cache->seq_lens;
    j.out = out;
    j.lse = lse;
    j.row_status = row_status;
    j.rows_of_head = FastDiv(static_cast<uint32_t>(rows * group));
    // sixteen columns a thread where there are more threads than the SMs hold at once
    const int64_t fours = static_cast<int64_t>(batch) * rows * q_heads * (cache->head_dim / 4);
    const bool many = fours > static_cast<int64_t>(h->sm_count) * 1024;
    j.columns = FastDiv(static_cast<uint32_t>(cache->head_dim / (many ? 16 : 4)));
    j.group = own.group;
    j.all = many ? fours / 4 : fours;
    j.batch = batch;
    j.heads = cache->kv_heads;
    j.rows = rows;
    j.q_heads = q_heads;
    j.dim = cache->head_dim;
    j.blocks = static_cast<int>((j.all + kPrefixJoinThreads - 1) / kPrefixJoinThreads);
    DeviceGuard g(h->device);
    if (!g.ok) return cuda_fail(cudaErrorInvalidDevice, "cudaSetDevice");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = beside ? p.own->launch(own, p.own_ctas, s) : p.prefix->launch(all, p.prefix_ctas, s);
    if (e == cudaSuccess) e = beside ? p.prefix->launch(all, p.prefix_ctas, s) : p.own->launch(own, p.own_ctas, s);
    const unsigned grid = static_cast<unsigned>(j.blocks + (batch + kPrefixJoinThreads - 1) / kPrefixJoinThreads);
    if (e == cudaSuccess)
        e = launch_early(cache->dtype == SPECV_BF16 ? prefix_join<__nv_bfloat16>(many) : prefix_join<float>(many), dim3(grid),
                         kPrefixJoinThreads, 0, s, j);
    if (e != cudaSuccess) return cuda_fail(e, "prefix_attention launch");
    h->launches.fetch_add(3, std::memory_order_relaxed);
    return SPECV_OK;
}

}  // extern "C"
