// prefix_attention.cuh -- attention of a batch whose sequences share a long
// prefix of the paged cache, which is read once for all of them.
//
// A row's softmax over prefix and own positions joins from the two parts'
// maxima, sums and weighted values (tree_attention.cuh).  The prefix is a
// part with one sequence whose rows are those of the whole batch, the own
// positions one with a sequence each: two launches of the kernels of tree
// attention, which leave every segment's results undivided in the workspace,
// and one that joins them.  The second launch does not wait for the first, only
// at its end; where both are tcgen05 kernels they share the SMs
// (tree_attention_tc.cuh).
//
// Measured (GB300, graph replays over sets of inputs beyond the L2; 32/8 heads of
// 128 in bf16; of 1896 TFLOP/s and 6803 GB/s measured):
//   64 single rows behind 4096 positions, 250..500 of their own   58.8 us, 29%
//   64 trees of 17 rows behind 8192, 500..1000                    171 us, 49%
//   16 chains of 6 rows behind 65536, 250..500                    104 us, 53%
//   fp32, 8 chains of 5, 12 heads of 64, behind 1024, 150..300    32 us, 8%
//   (heads of 64: trees 145 us, chains 92)
// On mma.sync, whose row tiles each read the prefix again: heads of 256 (16/4) single
// rows 84 us (bytes 17), trees 1170 (products 84), chains 710 (55); fp32, 16 trees of 17
// rows, 16/4 heads of 128, behind 4096 416 us (bytes 10.5).
// (the second by tree attention over all of its positions reads 2.3 GB).  The prefix
// of the trees alone takes 108 us, 70% of the tensor cores' rate, where the
// streams' turns bound it; their own positions alone 50; the join, some 12, and the
// short calls by latency.
#pragma once
#include "tree_attention.cuh"

namespace specv {

constexpr int kPrefixJoinThreads = 128;

// Of one of the two parts, for the join.
struct PartView {
    unsigned char* workspace;
    int64_t segs;
    int ctas, tm, row_tiles, dp;
    int side;     // from a CTA with a segment's piece to the next
    FastDiv tile;  // by tm
};

struct PrefixJoinArgs {
    PartView prefix, own;
    const int32_t* lens;
    void* out;
    float* lse;
    int32_t* row_status;
    FastDiv rows_of_head;  // rows * group
    FastDiv columns;       // a thread's columns of a head
    FastDiv group;
    int64_t all;  // threads: batch * kv heads * columns * rows * group
    int batch, heads, rows, q_heads, dim;
    int blocks;  // of the threads; behind them those that write the status
};

// The parts of a row joined so far, of COLS groups of four columns.
template <int COLS>
struct PrefixSum {
    float m = -INFINITY, l = 0.0f;
    float4 x[COLS];
    int status = 0;
};

// The pieces of segment `seg`, row `row` of its tile, columns 4 col ..; PIECES of them in flight.
template <int COLS, int PIECES>
__device__ __forceinline__ void prefix_join_part(const PartView& p, const PartNote& note, int64_t seg, int row, int col,
                                                 PrefixSum<COLS>& sum) {
    const PartWork work = part_work(p.workspace, p.ctas, p.segs, p.tm, p.dp);
    for (int c = note.first; c <= note.last; c += PIECES * p.side) {
        float2 ml[PIECES];
        float4 y[PIECES][COLS];
        int status[PIECES];
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            ml[u] = make_float2(-INFINITY, 0.0f);
            status[u] = 0;
#pragma unroll
            for (int k = 0; k < COLS; ++k) y[u][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const int at = c + u * p.side;
            if (at > note.last) continue;
            // whole; or [1] of the CTA that starts the segment, then [0] of the next ones
            const int64_t piece = note.first == note.last ? 2ll * p.ctas + seg : 2ll * at + (at == note.first);
            status[u] = work.status[piece];
            ml[u] = work.ml[piece * p.tm + row];
#pragma unroll
            for (int k = 0; k < COLS; ++k) y[u][k] = work.acc[(piece * (p.dp / 4) + col + k) * p.tm + row];
        }
        float m = sum.m;
#pragma unroll
        for (int u = 0; u < PIECES; ++u) m = fmaxf(m, ml[u].x);
        const float m_use = m == -INFINITY ? 0.0f : m;
        const float before = ex2(sum.m - m_use);
        sum.m = m;
        sum.l *= before;
#pragma unroll
        for (int k = 0; k < COLS; ++k)
            sum.x[k] = make_float4(sum.x[k].x * before, sum.x[k].y * before, sum.x[k].z * before, sum.x[k].w * before);
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            if (c + u * p.side > note.last) break;
            sum.status |= status[u];
            const float w = ex2(ml[u].x - m_use);
            sum.l = fmaf(ml[u].y, w, sum.l);
#pragma unroll
            for (int k = 0; k < COLS; ++k)
                sum.x[k] = make_float4(fmaf(y[u][k].x, w, sum.x[k].x), fmaf(y[u][k].y, w, sum.x[k].y),
                                       fmaf(y[u][k].z, w, sum.x[k].z), fmaf(y[u][k].w, w, sum.x[k].w));
        }
    }
}

__device__ __forceinline__ PartNote prefix_note(const PartView& p, int64_t seg) {
    return part_work(p.workspace, p.ctas, p.segs, p.tm, p.dp).segs[seg];
}

// Status bits of a segment's pieces, of every `step`-th from the `start`-th on.
__device__ __forceinline__ int prefix_status(const PartView& p, int64_t seg, int start, int step) {
    const PartWork work = part_work(p.workspace, p.ctas, p.segs, p.tm, p.dp);
    const PartNote note = work.segs[seg];
    int status = 0;
    for (int c = note.first + start * p.side; c <= note.last; c += step * p.side)
        status |= work.status[note.first == note.last ? 2ll * p.ctas + seg : 2ll * c + (c == note.first)];
    return status;
}

// A sequence's status: its first head's, that head's of the prefix, and waits
// that ran out.  A thread a sequence; what is the same for all is looked at by the CTA.
__device__ __forceinline__ void prefix_join_status(const PrefixJoinArgs& a, int b) {
    const AttnNote* prefix = reinterpret_cast<const AttnNote*>(a.prefix.workspace);
    const AttnNote* own = reinterpret_cast<const AttnNote*>(a.own.workspace);
    int late = 0;  // 1: a wait of the prefix's, 2: of the own part's CTAs
    for (int c = threadIdx.x; c < a.prefix.ctas; c += kPrefixJoinThreads) late |= prefix[c].failed != 0;
    for (int c = threadIdx.x; c < a.own.ctas; c += kPrefixJoinThreads) late |= own[c].failed != 0 ? 2 : 0;
    const int before = prefix_status(a.prefix, 0, threadIdx.x, kPrefixJoinThreads);
    __shared__ int s_late, s_before;
    if (threadIdx.x == 0) s_late = s_before = 0;
    __syncthreads();
    if (late) atomicOr(&s_late, late);
    if (before) atomicOr(&s_before, before);
    __syncthreads();
    if (b >= a.batch) return;
    int status = 0;
    if (a.lens[b] != 0) {
        status = prefix_status(a.own, static_cast<int64_t>(b) * a.heads * a.own.row_tiles, 0, 1);
        if (!(status & KV_LENGTH)) status |= s_before;  // (a sequence of a bad length is not looked at any further)
        if (s_late & 1) status |= KV_TIMEOUT;
        if (s_late & 2)
            for (int c = 0; c < a.own.ctas; ++c)
                if (own[c].failed && own[c].b0 <= b && b <= own[c].b1) status |= KV_TIMEOUT;
    }
    a.row_status[b] = status;
}

// COLS groups of four columns of a row a thread, rows of a kv head side by
// side.  Bound by latency (length, notes, pieces, one behind the other): a
// thread has many pieces in flight where there are few rows, each spread over
// many CTAs, and many columns where there are many, in two or three pieces.
template <typename T, int COLS, int PIECES>
__global__ void __launch_bounds__(kPrefixJoinThreads) prefix_join_kernel(const PrefixJoinArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x >= a.blocks) {
        if (a.row_status) prefix_join_status(a, (blockIdx.x - a.blocks) * kPrefixJoinThreads + threadIdx.x);
        return;
    }
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kPrefixJoinThreads + threadIdx.x;
    if (at >= a.all) return;
    // rows of a head fastest, then columns, heads, sequences (the quotients below 2^31: `all` is)
    const uint32_t i = static_cast<uint32_t>(at);
    const uint32_t x = a.rows_of_head.div(i), m = i - x * a.rows_of_head.d;
    const uint32_t y = a.columns.div(x), col = (x - y * a.columns.d) * COLS;
    const int b = static_cast<int>(y / static_cast<uint32_t>(a.heads)), h = static_cast<int>(y) - b * a.heads;
    const uint32_t r = a.group.div(m), g = m - r * a.group.d;
    const uint32_t own_tile = a.own.tile.div(m);
    const int64_t own_seg = (static_cast<int64_t>(b) * a.heads + h) * a.own.row_tiles + own_tile;
    const uint32_t row = static_cast<uint32_t>(b) * a.rows_of_head.d + m, tile = a.prefix.tile.div(row);
    const int64_t seg = static_cast<int64_t>(h) * a.prefix.row_tiles + tile;
    const PartNote own_note = prefix_note(a.own, own_seg), note = prefix_note(a.prefix, seg);
    PrefixSum<COLS> sum;
#pragma unroll
    for (int k = 0; k < COLS; ++k) sum.x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const bool idle = a.lens[b] == 0;
    if (!idle) {
        prefix_join_part<COLS, COLS == 1 ? 8 : 2>(a.own, own_note, own_seg, m - own_tile * a.own.tm, col, sum);
        prefix_join_part<COLS, PIECES>(a.prefix, note, seg, row - tile * a.prefix.tm, col, sum);
    }
    const bool zero = idle || sum.status != 0;
    const float inv = zero ? 0.0f : 1.0f / sum.l;
    const int64_t head = (static_cast<int64_t>(b) * a.rows + r) * a.q_heads + static_cast<int64_t>(h) * a.group.d + g;
#pragma unroll
    for (int k = 0; k < COLS; ++k) {
        if (zero) sum.x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        attn_store4(static_cast<T*>(a.out) + head * a.dim + (col + k) * 4, sum.x[k].x * inv, sum.x[k].y * inv,
                    sum.x[k].z * inv, sum.x[k].w * inv);
    }
    if (col == 0 && a.lse) a.lse[head] = zero ? -INFINITY : sum.m * 0.693147181f + logf(sum.l);
}

}  // namespace specv
