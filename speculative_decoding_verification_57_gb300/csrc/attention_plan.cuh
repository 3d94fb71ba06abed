// attention_plan.cuh -- which kernel an attention call takes, by type, head
// size and rows, and its launch.
#pragma once
#include "cache_host.cuh"
#include "tree_attention.cuh"
#include "tensor_maps.cuh"

namespace {

// The join behind tree attention of one shape.
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

// A part's results are joined with those of another.
template <typename S>
cudaError_t launch_join(const PartArgs&, int, cudaStream_t) {
    return cudaSuccess;
}

template <typename S, typename A>
cudaError_t launch_attention(const A& a, int ctas, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(tree_attention_kernel<S, A>), S::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_early(tree_attention_kernel<S, A>, dim3(static_cast<unsigned>(ctas)), S::kThreads, S::kSmem, stream, a);
    return e != cudaSuccess ? e : launch_join<S>(a, ctas, stream);
}

// Boxes for the cache's blocks, and for the queries where these fill row tiles.
bool make_maps(const AttnArgs& a, TcMaps& maps) {
    const TensorMapEncode encode = tensor_map_encode();
    if (!encode || !make_pool_maps(a.kv, maps)) return false;
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    // the queries, a row tile a box and panel, where groups of heads fill row tiles
    const int group = static_cast<int>(a.group.d);
    maps.q_rows = 0;
    if (128 % group == 0 && a.q_stride > 0 && a.q_stride * a.rows < (1ll << 38)) {
        const cuuint64_t q_dims[4] = {static_cast<cuuint64_t>(a.kv.dim), static_cast<cuuint64_t>(a.q_heads), static_cast<cuuint64_t>(a.rows),
                                      static_cast<cuuint64_t>(a.batch)};
        const cuuint64_t q_strides[3] = {static_cast<cuuint64_t>(a.kv.dim) * 2, static_cast<cuuint64_t>(a.q_stride) * 2,
                                         static_cast<cuuint64_t>(a.q_stride) * a.rows * 2};
        const cuuint32_t q_box[4] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(128 / group), 1};
        if (encode(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.q), q_dims, q_strides, q_box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS)
            maps.q_rows = 128 / group;
    }
    return true;
}

template <typename S, typename A>
cudaError_t launch_tc(const A& a, const TcMaps& maps, int ctas, cudaStream_t stream) {
    constexpr int kBytes = sizeof(TcShared<S>);
    static_assert(kBytes <= 227 * 1024, "a CTA's shared memory");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(tree_attention_tc_kernel<S, A>), kBytes);
    if (e != cudaSuccess) return e;
    e = launch_early(tree_attention_tc_kernel<S, A>, dim3(static_cast<unsigned>(ctas)), S::kThreads, kBytes, stream, a, maps);
    return e != cudaSuccess ? e : launch_join<S>(a, ctas, stream);
}

template <int DP, bool WIDE, typename A, int BOXES = 2>
cudaError_t launch_attention_tc(const A& a, int ctas, cudaStream_t stream) {
    TcMaps maps = {};
    if (make_maps(a, maps)) return launch_tc<TcShape<DP, WIDE, true, BOXES>, A>(a, maps, ctas, stream);
    return launch_tc<TcShape<DP, WIDE, false>, A>(a, maps, ctas, stream);
}

template <typename A>
struct AttnPlan {
    int dp, tm, ctas;  // padded head_dim, rows of a tile, CTAs an SM
    bool tc;           // the tcgen05 kernel
    cudaError_t (*launch)(const A&, int, cudaStream_t);
};

template <typename A, typename S>
constexpr AttnPlan<A> plan_of() {
    return AttnPlan<A>{S::DP, S::TM, S::kCtas, false, launch_attention<S, A>};
}

template <typename A, int DP, bool WIDE>
constexpr AttnPlan<A> plan_of_tc() {
    return AttnPlan<A>{DP, TcShape<DP, WIDE, true>::TM, 1, true, launch_attention_tc<DP, WIDE, A>};
}

// bf16 rows up to head_dim 128 and more than 16 rows a kv head (rows * group)
// go to the tcgen05 kernel, whose row tile of 128 costs the tensor cores less
// time than its positions cost the memory; up to 16 the other's pipeline is
// shorter.  Single rows, 32/8 heads of 128, this kernel | the tcgen05 one, us:
//   sequences   500 positions   2000          20,000        131,072
//   1           9.2 | 10.6      15.1 | 14.1   29.8 | 27.4   101 | 93
//   4           10.5 | 12.5     16.9 | 18.4   53.4 | 50.7   283 | 261
//   64          33.1 | 40.6     79.5 | 75.4   605 | 562
// 16 heads of 64, 128 single rows over 1000 positions 92 | 139, 16 rows for 64
// over 2000 87 | 104, for 4 over 20,000 56 | 61.  So long contexts of heads of 128
// would be 5 to 8% faster
// there; but lengths are device memory, and the rule does not look at them.  Of
// 20 rows a kv head, 64 sequences over 300 positions took 42.3 us on this
// kernel (with a row tile of 32) and take 33.4 there, 1 over 2000 13.7 and 14.3.  In
// each, the narrowest row tile that holds the rows, or the widest: a tile's
// keys and values are read once for all of its rows.
constexpr int kTcLeast = 17;

template <typename A>
const AttnPlan<A>& attn_plan(specv_dtype dt, int dim, int m) {
    using B = __nv_bfloat16;
    using F = float;
    static constexpr AttnPlan<A> f32[3][3] = {
        {plan_of<A, AttnShape<F, 64, 1, 1>>(), plan_of<A, AttnShape<F, 64, 1, 2>>(), plan_of<A, AttnShape<F, 64, 2, 2>>()},
        {plan_of<A, AttnShape<F, 128, 1, 1>>(), plan_of<A, AttnShape<F, 128, 1, 2>>(), plan_of<A, AttnShape<F, 128, 2, 2>>()},
        {plan_of<A, AttnShape<F, 256, 1, 1>>(), plan_of<A, AttnShape<F, 256, 1, 2>>(), plan_of<A, AttnShape<F, 256, 1, 2>>()}};
    static constexpr AttnPlan<A> few[2] = {plan_of<A, AttnShape<B, 64, 1, 1>>(), plan_of<A, AttnShape<B, 128, 1, 1>>()};
    static constexpr AttnPlan<A> many[2][2] = {{plan_of_tc<A, 64, false>(), plan_of_tc<A, 64, true>()},
                                            {plan_of_tc<A, 128, false>(), plan_of_tc<A, 128, true>()}};
    static constexpr AttnPlan<A> big[2] = {plan_of<A, AttnShape<B, 256, 1, 1>>(), plan_of<A, AttnShape<B, 256, 1, 2>>()};
    const int d = dim <= 64 ? 0 : dim <= 128 ? 1 : 2;
    if (dt == SPECV_F32) return f32[d][m <= 16 ? 0 : m <= 32 ? 1 : 2];
    if (d == 2) return big[m <= 16 ? 0 : 1];
    return m < kTcLeast ? few[d] : many[d][m <= 128 ? 0 : 1];
}

// The prefix's part in row tiles of 128 side by side (bf16, head_dim up to 128).
inline const AttnPlan<PartArgs>& side_plan(int dim) {
    static constexpr AttnPlan<PartArgs> plans[2] = {{64, 128, 1, true, launch_attention_tc<64, false, PartArgs, 3>},
                                                    {128, 128, 1, true, launch_attention_tc<128, false, PartArgs, 3>}};
    return plans[dim <= 64 ? 0 : 1];
}

}  // namespace
