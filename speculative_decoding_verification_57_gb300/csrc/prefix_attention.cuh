// prefix_attention.cuh -- attention of a batch whose sequences share a long
// prefix of the paged cache, which is read once for all of them.
//
// A row's softmax over prefix and own positions joins from the two parts'
// maxima, sums and weighted values (tree_attention.cuh).  The prefix is a
// part with one sequence whose rows are those of the whole batch, the own
// positions one with a sequence each: two launches of the kernels of tree
// attention, which leave every segment's results undivided in the workspace,
// and one that joins them.
#pragma once
#include "tree_attention.cuh"

namespace specv {

constexpr int kPrefixJoinThreads = 128;

// Of one of the two parts, for the join.
struct PartView {
    unsigned char* workspace;
    int64_t segs;
    int ctas, tm, row_tiles, dp;
    FastDiv tile;  // by tm
};

struct PrefixJoinArgs {
    PartView prefix, own;
    const int32_t* lens;
    void* out;
    float* lse;
    int32_t* row_status;
    FastDiv rows_of_head;  // rows * group
    FastDiv columns;       // groups of four columns of a head
    FastDiv group;
    int64_t all;  // threads: batch * kv heads * columns * rows * group
    int batch, heads, rows, q_heads, dim;
    int blocks;  // of the threads; behind them those that write the status
};

// The parts of a row joined so far.
struct PrefixSum {
    float m = -INFINITY, l = 0.0f;
    float4 x = {0.0f, 0.0f, 0.0f, 0.0f};
    int status = 0;
};

// The pieces of segment `seg`, row `row` of its tile, columns 4 col ..
__device__ __forceinline__ void prefix_join_part(const PartView& p, int64_t seg, int row, int col, PrefixSum& sum) {
    const PartWork work = part_work(p.workspace, p.ctas, p.segs, p.tm, p.dp);
    const PartNote note = work.segs[seg];
    constexpr int kPieces = 4;  // in flight
    for (int c = note.first; c <= note.last; c += kPieces) {
        float2 ml[kPieces];
        float4 y[kPieces];
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            ml[u] = make_float2(-INFINITY, 0.0f);
            y[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c + u > note.last) continue;
            // whole; or [1] of the CTA that starts the segment, then [0] of the next ones
            const int64_t piece = note.first == note.last ? 2ll * p.ctas + seg : 2ll * (c + u) + (c + u == note.first);
            sum.status |= work.status[piece];
            ml[u] = work.ml[piece * p.tm + row];
            y[u] = work.acc[(piece * (p.dp / 4) + col) * p.tm + row];
        }
        float m = sum.m;
#pragma unroll
        for (int u = 0; u < kPieces; ++u) m = fmaxf(m, ml[u].x);
        const float m_use = m == -INFINITY ? 0.0f : m;
        const float before = ex2(sum.m - m_use);
        sum.m = m;
        sum.l *= before;
        sum.x = make_float4(sum.x.x * before, sum.x.y * before, sum.x.z * before, sum.x.w * before);
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            if (c + u > note.last) break;
            const float w = ex2(ml[u].x - m_use);
            sum.l = fmaf(ml[u].y, w, sum.l);
            sum.x = make_float4(fmaf(y[u].x, w, sum.x.x), fmaf(y[u].y, w, sum.x.y), fmaf(y[u].z, w, sum.x.z),
                                fmaf(y[u].w, w, sum.x.w));
        }
    }
}

// Status bits of a segment's pieces.
__device__ __forceinline__ int prefix_status(const PartView& p, int64_t seg) {
    const PartWork work = part_work(p.workspace, p.ctas, p.segs, p.tm, p.dp);
    const PartNote note = work.segs[seg];
    if (note.first == note.last) return work.status[2ll * p.ctas + seg];
    int status = 0;
    for (int c = note.first; c <= note.last; ++c) status |= work.status[2ll * c + (c == note.first)];
    return status;
}

// Four columns of a row a thread, rows of a kv head side by side.
template <typename T>
__global__ void __launch_bounds__(kPrefixJoinThreads) prefix_join_kernel(const PrefixJoinArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x >= a.blocks) {  // a sequence's status: its first head's, that head's of the prefix, and waits that ran out
        if (!a.row_status) return;
        const int b = (blockIdx.x - a.blocks) * kPrefixJoinThreads + threadIdx.x;
        const AttnNote* prefix = reinterpret_cast<const AttnNote*>(a.prefix.workspace);
        const AttnNote* own = reinterpret_cast<const AttnNote*>(a.own.workspace);
        bool late = false;
        for (int c = threadIdx.x; c < a.prefix.ctas; c += kPrefixJoinThreads) late |= prefix[c].failed != 0;
        late = __syncthreads_or(late) != 0;
        if (b >= a.batch) return;
        int status = 0;
        if (a.lens[b] != 0) {
            status = prefix_status(a.own, static_cast<int64_t>(b) * a.heads * a.own.row_tiles);
            // (a sequence of a bad length is not looked at any further; the prefix's table is the same for every head)
            if (!(status & KV_LENGTH)) status |= prefix_status(a.prefix, 0);
            if (late) status |= KV_TIMEOUT;
            for (int c = 0; c < a.own.ctas; ++c)
                if (own[c].failed && own[c].b0 <= b && b <= own[c].b1) status |= KV_TIMEOUT;
        }
        a.row_status[b] = status;
        return;
    }
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kPrefixJoinThreads + threadIdx.x;
    if (at >= a.all) return;
    // rows of a head fastest, then columns, heads, sequences (the quotients below 2^31: `all` is)
    const uint32_t i = static_cast<uint32_t>(at);
    const uint32_t x = a.rows_of_head.div(i), m = i - x * a.rows_of_head.d;
    const uint32_t y = a.columns.div(x), col = x - y * a.columns.d;
    const int b = static_cast<int>(y / static_cast<uint32_t>(a.heads)), h = static_cast<int>(y) - b * a.heads;
    const uint32_t r = a.group.div(m), g = m - r * a.group.d;
    PrefixSum sum;
    const bool idle = a.lens[b] == 0;
    if (!idle) {
        const uint32_t mine = a.own.tile.div(m);
        prefix_join_part(a.own, (static_cast<int64_t>(b) * a.heads + h) * a.own.row_tiles + mine, m - mine * a.own.tm, col,
                         sum);
        const uint32_t row = static_cast<uint32_t>(b) * a.rows_of_head.d + m, tile = a.prefix.tile.div(row);
        prefix_join_part(a.prefix, static_cast<int64_t>(h) * a.prefix.row_tiles + tile, row - tile * a.prefix.tm, col, sum);
    }
    const bool zero = idle || sum.status != 0;
    const float inv = zero ? 0.0f : 1.0f / sum.l;
    if (zero) sum.x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int64_t head = (static_cast<int64_t>(b) * a.rows + r) * a.q_heads + static_cast<int64_t>(h) * a.group.d + g;
    attn_store4(static_cast<T*>(a.out) + head * a.dim + col * 4, sum.x.x * inv, sum.x.y * inv, sum.x.z * inv,
                sum.x.w * inv);
    if (col == 0 && a.lse) a.lse[head] = zero ? -INFINITY : sum.m * 0.693147181f + logf(sum.l);
}

}  // namespace specv
