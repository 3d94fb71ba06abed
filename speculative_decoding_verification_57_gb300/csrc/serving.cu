// serving.cu -- C ABI of the calls on the paged KV cache for current models
// and long-running batches: append with head norms and positions on axes,
// the attention weight that positions gather, and eviction by it.  A
// translation unit of its own, compiled beside library.cu.
#include <cmath>

#include "append_norm.cuh"
#include "attention_mass_tc.cuh"
#include "cache_evict.cuh"
#include "cache_host.cuh"
#include "tensor_maps.cuh"

namespace {

using NormKernel = void (*)(AppendNormArgs);

template <typename T, int THREADS>
NormKernel norm_kernel_of(int mode) {
    return mode == kApart        ? cache_append_norm_kernel<T, kApart, THREADS>
           : mode == kNeighbours ? cache_append_norm_kernel<T, kNeighbours, THREADS>
                                 : cache_append_norm_kernel<T, kValues, THREADS>;
}

NormKernel norm_kernel(specv_dtype dt, int mode, bool many) {
    using B = __nv_bfloat16;
    if (dt == SPECV_BF16) return many ? norm_kernel_of<B, kAppendMany>(mode) : norm_kernel_of<B, kAppendFew>(mode);
    return many ? norm_kernel_of<float, kAppendMany>(mode) : norm_kernel_of<float, kAppendFew>(mode);
}

template <typename T, int DP, int NT>
cudaError_t launch_mass_of(const MassArgs& a, int sms, cudaStream_t stream) {
    using S = MassShape<T, DP, NT>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(attention_mass_kernel<S>), S::kSmem);
    if (e != cudaSuccess) return e;
    return launch_early(attention_mass_kernel<S>, dim3(static_cast<unsigned>(sms * S::kCtas)), S::kThreads, S::kSmem, stream,
                        a);
}

// Ten tiles of eight queries at a time, in turns, or the fewest of one, four and ten that hold a kv head's: what a tile costs is
// formed for all of them.  In one, four and ten tiles, us: fp32, 32 sequences over 1000..2000 positions, 32/8 heads of 128,
// 8 queries a kv head 63, 146, 273, 32 queries 160 in four and 302 in ten, 68 queries 403 and 301; bf16, 64 sequences, 16/4
// heads of 256, 8 queries 48, 78, 97, 32 queries 83 and 102, 68 queries 202 and 119 (bytes alone: 28.6).
template <typename T, int DP>
cudaError_t launch_mass(const MassArgs& a, int sms, cudaStream_t stream) {
    if constexpr (sizeof(T) == 4 || DP > 128) {
        const int m = a.rows * static_cast<int>(a.group.d);
        if (m <= 8) return launch_mass_of<T, DP, 1>(a, sms, stream);
        if (m <= 32) return launch_mass_of<T, DP, 4>(a, sms, stream);
    }
    return launch_mass_of<T, DP, 10>(a, sms, stream);
}

template <typename S>
cudaError_t launch_mass_tc_of(const MassArgs& a, const TcMaps& maps, int sms, cudaStream_t stream) {
    constexpr int kBytes = sizeof(MassShared<S>);
    static_assert(kBytes <= 227 * 1024, "a CTA's shared memory");
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(attention_mass_tc_kernel<S>), kBytes);
    if (e != cudaSuccess) return e;
    return launch_early(attention_mass_tc_kernel<S>, dim3(static_cast<unsigned>(sms)), S::kThreads, kBytes, stream, a, maps);
}

template <int DP>
cudaError_t launch_mass_tc(const MassArgs& a, int sms, cudaStream_t stream) {
    TcMaps maps = {};
    if (make_pool_maps(a.kv, maps)) return launch_mass_tc_of<MassTc<DP, true>>(a, maps, sms, stream);
    return launch_mass_tc_of<MassTc<DP, false>>(a, maps, sms, stream);
}

// bf16, head_dim up to 128 and up to 256 queries a kv head go to the tcgen05
// kernel (64 single rows of 32/8 heads of 128 over 1000..2000 positions 40 us, on
// the other 48; trees of 17 rows over 2048..4096 78 and 276).
bool mass_tc(specv_dtype dt, const MassArgs& a) {
    return dt == SPECV_BF16 && a.kv.dim <= 128 && a.rows * static_cast<int>(a.group.d) <= 256;
}

cudaError_t launch_mass_tc(const MassArgs& a, int sms, cudaStream_t stream) {
    return a.kv.dim <= 64 ? launch_mass_tc<64>(a, sms, stream) : launch_mass_tc<128>(a, sms, stream);
}

template <typename T>
cudaError_t launch_mass(const MassArgs& a, int sms, cudaStream_t stream) {
    if (a.kv.dim <= 64) return launch_mass<T, 64>(a, sms, stream);
    if (a.kv.dim <= 128) return launch_mass<T, 128>(a, sms, stream);
    return launch_mass<T, 256>(a, sms, stream);
}

// Whether `m` bytes at p and `n` bytes at q have any in common.
bool overlap(const void* p, int64_t m, const void* q, int64_t n) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + static_cast<uintptr_t>(n) && b < a + static_cast<uintptr_t>(m);
}

}  // namespace

extern "C" {

specv_status specv_cache_append_norm(specv_handle h, const specv_kv_cache* cache, const void* q, int64_t q_stride,
                                     int q_heads, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                     const specv_head_norm* norm, const float* inv_freq, int rot_dim, int interleaved,
                                     const specv_positions* positions, const int32_t* parents,
                                     const int32_t* row_counts, int batch, int rows, void* q_out, int32_t* row_status,
                                     void* stream) {
    AppendNormArgs n = {};
    AppendArgs& a = n.a;
    if (!make_view(h, cache, batch, a.kv)) return SPECV_ERR_INVALID_ARGUMENT;
    if (rows < 1 || (parents && rows - 1 > h->max_k)) return SPECV_ERR_INVALID_ARGUMENT;
    if (static_cast<int64_t>(batch) * rows > INT32_MAX) return SPECV_ERR_INVALID_ARGUMENT;
    if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 2 || (rot_dim > 0 && !inv_freq))
        return SPECV_ERR_INVALID_ARGUMENT;
    if (norm) {
        if (!std::isfinite(norm->eps) || norm->eps < 0.0f || !std::isfinite(norm->weight_add) ||
            !aligned16(norm->q_weight) || !aligned16(norm->k_weight))
            return SPECV_ERR_INVALID_ARGUMENT;
        n.q_weight = norm->q_weight;
        n.k_weight = norm->k_weight;
        n.eps = norm->eps;
        n.weight_add = norm->weight_add;
    }
    if (positions && positions->positions) {
        if (positions->axes < 1 || positions->axes > 16 || positions->offsets || parents) return SPECV_ERR_INVALID_ARGUMENT;
        if (positions->axes > 1 && rot_dim > 0 && !positions->pair_axis) return SPECV_ERR_INVALID_ARGUMENT;
        n.positions = positions->positions;
        n.axes = positions->axes;
        for (int j = 0; j < rot_dim / 2; ++j) {
            n.axis[j] = positions->pair_axis ? positions->pair_axis[j] : 0;
            if (n.axis[j] >= n.axes) return SPECV_ERR_INVALID_ARGUMENT;
        }
    } else if (positions) {
        n.offsets = positions->offsets;
    }
    // nothing that the plain append does not do
    if (!n.q_weight && !n.k_weight && !n.positions && !n.offsets)
        return specv_cache_append(h, cache, q, q_stride, q_heads, k, k_stride, v, v_stride, inv_freq, rot_dim, interleaved,
                                  parents, row_counts, batch, rows, q_out, row_status, stream);
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
    const int units = cache->head_dim / vec / 2;
    a.units = FastDiv(static_cast<uint32_t>(units));
    while ((1 << n.group_log) < units) ++n.group_log;
    n.inv_dim = 1.0f / static_cast<float>(cache->head_dim);
    DeviceGuard g(h->device);
    if (!g.ok) return cuda_fail(cudaErrorInvalidDevice, "cudaSetDevice");
    const unsigned grid = static_cast<unsigned>(batch) * static_cast<unsigned>(rows);
    const bool many = grid > static_cast<unsigned>(h->sm_count) * (kNormResident / kAppendFew);
    // pieces of 16 bytes turn whole, apart or within, where rot_dim fills them
    const int mode = rot_dim % (interleaved ? vec : 2 * vec) ? kValues : interleaved && rot_dim ? kNeighbours : kApart;
    const NormKernel kernel = norm_kernel(cache->dtype, mode, many);
    kernel<<<grid, many ? kAppendMany : kAppendFew, 0, static_cast<cudaStream_t>(stream)>>>(n);
    return launched(h, "cache_append_norm launch");
}

specv_status specv_attention_mass(specv_handle h, const specv_kv_cache* cache, const void* q, int64_t q_stride,
                                  int q_heads, const int32_t* parents, int batch, int rows, float scale,
                                  const float* lse, const int32_t* path, const int32_t* num_accepted,
                                  const float* mass, float* mass_out, int64_t width, int first, int32_t* row_status,
                                  void* stream) {
    MassArgs a = {};
    if (!make_view(h, cache, batch, a.kv)) return SPECV_ERR_INVALID_ARGUMENT;
    if (rows < 1 || rows - 1 > h->max_k || q_heads < 1 || q_heads > 65536 || q_heads % cache->kv_heads ||
        !std::isfinite(scale) || !std::isfinite(attn_scale(scale)) || width < 0 || width > INT32_MAX || first < 0)
        return SPECV_ERR_INVALID_ARGUMENT;
    if (batch == 0) return SPECV_OK;
    if (!rows_ok(cache, q, q_stride) || !lse || (width > 0 && !mass_out)) return SPECV_ERR_INVALID_ARGUMENT;
    const int64_t mass_bytes = static_cast<int64_t>(batch) * cache->kv_heads * width * 4;
    if (mass && mass != mass_out && overlap(mass, mass_bytes, mass_out, mass_bytes)) return SPECV_ERR_INVALID_ARGUMENT;
    a.q = q;
    a.q_stride = q_stride;
    a.parents = rows > 1 ? parents : nullptr;
    a.lse = lse;
    a.path = num_accepted ? path : nullptr;
    a.num_accepted = num_accepted;
    a.mass = mass;
    a.out = mass_out;
    a.row_status = row_status;
    a.width = width;
    a.group = FastDiv(static_cast<uint32_t>(q_heads / cache->kv_heads));
    a.q_heads = q_heads;
    a.rows = rows;
    a.batch = batch;
    a.row_tiles = 1;
    a.first = first;
    a.skip = first / cache->block_size * cache->block_size;
    a.scale = scale;
    a.withhold = -1;
    a.polls = 1u << 30;
    const bool tc = mass_tc(cache->dtype, a);
    if (tc && h->test_withhold >= 0) {  // the test hook arms one launch
        a.withhold = h->test_withhold;
        a.polls = h->test_polls;
        h->test_withhold = -1;
    }
    DeviceGuard g(h->device);
    if (!g.ok) return cuda_fail(cudaErrorInvalidDevice, "cudaSetDevice");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = tc                           ? launch_mass_tc(a, h->sm_count, s)
                          : cache->dtype == SPECV_BF16 ? launch_mass<__nv_bfloat16>(a, h->sm_count, s)
                                                       : launch_mass<float>(a, h->sm_count, s);
    if (e != cudaSuccess) return cuda_fail(e, "attention_mass launch");
    h->launches.fetch_add(1, std::memory_order_relaxed);
    return SPECV_OK;
}

specv_status specv_cache_evict(specv_handle h, const specv_kv_cache* cache, int layers, int64_t layer_stride,
                               const float* mass, float* mass_out, int64_t width, int batch, int budget, int recent,
                               int first, int32_t* lens_out, int32_t* evicted, int32_t* row_status, void* stream) {
    EvictArgs e = {};
    if (!make_view(h, cache, batch, e.kv)) return SPECV_ERR_INVALID_ARGUMENT;
    const int vec = cache->dtype == SPECV_BF16 ? 8 : 4;
    if (layers < 1 || layers > 65536 || layer_stride < 0 || layer_stride % vec || width < 0 || width > INT32_MAX)
        return SPECV_ERR_INVALID_ARGUMENT;
    if (layers > 1 && layer_stride < static_cast<int64_t>(cache->kv_heads) * cache->block_size * cache->head_dim)
        return SPECV_ERR_INVALID_ARGUMENT;
    if (layer_stride > INT64_MAX / 16 / layers) return SPECV_ERR_INVALID_ARGUMENT;
    if (budget < 1 || recent < 0 || first < 0 || static_cast<int64_t>(recent) + first > budget)
        return SPECV_ERR_INVALID_ARGUMENT;
    if (batch == 0) return SPECV_OK;
    const int64_t rows = static_cast<int64_t>(layers) * batch * cache->kv_heads;
    if (!lens_out || rows > INT32_MAX / 16) return SPECV_ERR_INVALID_ARGUMENT;
    // (every CTA of a sequence reads its length and its blocks, while one writes what the call tells of it)
    const int64_t entries = static_cast<int64_t>(batch) * cache->max_blocks;
    for (const int32_t* out : {lens_out, evicted, row_status})
        if (out && (overlap(out, batch * 4ll, cache->seq_lens, batch * 4ll) ||
                    overlap(out, batch * 4ll, cache->block_tables, entries * 4)))
            return SPECV_ERR_INVALID_ARGUMENT;
    if (width > 0 && (!mass || !mass_out || overlap(mass, rows * width * 4, mass_out, rows * width * 4)))
        return SPECV_ERR_INVALID_ARGUMENT;
    e.mass = mass;
    e.mass_out = mass_out;
    e.lens_out = lens_out;
    e.evicted = evicted;
    e.row_status = row_status;
    e.layer_stride = layer_stride;
    e.width = width;
    e.batch = batch;
    e.budget = budget;
    e.recent = recent;
    e.first = first;
    e.vec_elems = vec;
    // few rows: CTAs side by side for keys and values and for columns, of 32 bytes at least
    const int pieces = cache->head_dim / vec;
    e.split = 1;
    int columns = 1;
    if (rows < 4 * h->sm_count) {
        while (columns < 4 && pieces % (2 * columns) == 0 && pieces / columns >= 4 && rows * columns * 4 <= 4 * h->sm_count)
            columns *= 2;
        e.split = 2 * columns;
    }
    e.pieces = pieces / columns;
    e.piece_div = FastDiv(static_cast<uint32_t>(e.pieces));
    DeviceGuard g(h->device);
    if (!g.ok) return cuda_fail(cudaErrorInvalidDevice, "cudaSetDevice");
    cache_evict_kernel<<<static_cast<unsigned>(rows * e.split), kEvictThreads, 0, static_cast<cudaStream_t>(stream)>>>(e);
    return launched(h, "cache_evict launch");
}

}  // extern "C"
