// attention_mass.cuh -- the attention weight that the positions of a paged
// cache gather from a pass: mass[b, h, t] (+)= sum over the pass's rows r that
// see t and the query heads g of kv head h of exp(scale q.k_t - lse[b, r, g]).
//
// The softmax's sums are given (lse), so a position's weights need nothing of
// the others: tiles of KT positions are independent, each read once, and
// results need no joining and no atomics.  All sequences' tiles form one line,
// cut into equal runs on the device, one a CTA, as in tree_attention.cuh.  A
// warp has 16 MT positions as the rows of its matrix instructions and takes
// the queries eight columns each, so that a thread adds up the columns of its
// positions by itself and three shuffles finish a position.
//
// For fp32, heads above 128 and more than 256 queries a kv head; the rest is in
// attention_mass_tc.cuh.  fp32 is bound by the instructions that split keys and
// queries into tf32 parts, bf16 by the scores' way through registers.
//
// Measured (GB300, graph replays over sets of inputs beyond the L2; of 6803 GB/s): heads
// of 256 (16/4) in bf16, 64 single rows over 1000..2000 positions 49 us, 60%, trees of 17
// rows over 2048..4096 233 us, 26%; fp32, 32 sequences over 1000..2000, 32/8 heads of
// 128, single rows 63 us, 45%, trees of 17 rows 301 us, 10%; bf16, 32 rows of 9 query
// heads a kv head (288 queries) there 270 us, 6% (of 8, on tcgen05, 69).
#pragma once
#include "tree_attention.cuh"

namespace specv {

struct MassArgs {
    KvView kv;
    const void* q;
    int64_t q_stride;
    const int32_t* parents;
    const float* lse;   // [B, rows, q_heads]
    const float* mass;  // [B, heads, width]; NULL: zeros
    float* out;         // [B, heads, width]
    const int32_t *path, *num_accepted;  // of a verified pass (NULL: all rows stay)
    int32_t* row_status;
    int64_t width;
    FastDiv group;
    int q_heads, rows, batch;
    int row_tiles;  // 1
    int first;      // positions before it are left alone
    int skip;       // whole blocks before it, which are not read
    float scale;
    int withhold;    // test hook: copy of CTA 0 that never happens; -1: none
    uint32_t polls;  // most polls of a wait
};

// Positions of sequence b from `skip` on; 0: nothing to do; -1: refused by its length.
__device__ __forceinline__ int attn_len(const MassArgs& a, int b) {
    const int len = a.kv.lens[b];
    if (len == 0) return 0;
    if (len < a.rows || !a.kv.fits(len) || len > a.width) return -1;
    return len > a.skip ? len - a.skip : 0;
}

__device__ __forceinline__ int attn_side(const MassArgs&) { return 1; }

// What stays of sequence b's pass, by one converged warp; lane r holds row r.
// Returns the rows that stay (bit r: row 0, and a kept node's), and as `to` the
// row's place among the pass's positions behind them, -1 if it goes; `status`
// gets the bits of a count or a path that are none.
__device__ __forceinline__ uint32_t mass_kept(const MassArgs& a, int b, int lane, int& to, int& status) {
    to = lane < a.rows ? lane : -1;
    if (!a.num_accepted) return ~0u;
    const int nodes = a.rows - 1, n = a.num_accepted[b];
    if (n < 0 || n > nodes) status |= KV_ACCEPTED;
    const bool mine = lane < nodes && lane < n;
    const int node = mine ? a.path ? a.path[static_cast<int64_t>(b) * nodes + lane] : lane : -1;
    const int before = __shfl_up_sync(0xffffffffu, node, 1);
    if (!__all_sync(0xffffffffu, !mine || (node >= 0 && node < nodes && (lane == 0 || node > before)))) status |= KV_PATH;
    uint32_t kept = 1 | (mine && node >= 0 && node < nodes ? 2u << node : 0u);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) kept |= __shfl_xor_sync(0xffffffffu, kept, off);
    // (a path is increasing: a kept row's place is the number of kept rows above it)
    to = kept >> lane & 1 ? __popc(kept & ((1u << lane) - 1)) : -1;
    return kept;
}

// DP: head_dim rounded up to 64, 128 or 256; NT tiles of eight queries at a
// time; MT row groups of 16 positions a warp, four warps.
template <typename T, int DP_, int NT_>
struct MassShape {
    using Type = T;
    static constexpr bool kBf16 = sizeof(T) == 2;
    static constexpr int DP = DP_, NT = NT_;
    static constexpr int MT = kBf16 && DP <= 128 ? 2 : 1;
    static constexpr int KT = 64 * MT;
    static constexpr int kThreads = 128;
    static constexpr int kRow = DP * static_cast<int>(sizeof(T));
    static constexpr int kTile = KT * kRow;
    static constexpr int NQ = 8 * NT;  // queries at a time
    static constexpr int kQ = NQ * kRow;
    static constexpr int kStages = kTile > 48 * 1024 ? 2 : 3;
    static constexpr int kAhead = kStages - 1;
    static constexpr int kSmem = kStages * kTile + kQ;
    static constexpr int kFit = 227 * 1024 / (kSmem + 3 * 1024);
    // resident CTAs: by shared memory and by registers (scores, and some 70 others)
    static constexpr int kMost = 65536 / ((MT * NT * (kBf16 ? 4 : 8) + 70) * kThreads);
    static constexpr int kCtas = kFit > kMost ? kMost : kFit;
};

template <typename S>
__global__ void __launch_bounds__(S::kThreads, S::kCtas) attention_mass_kernel(const MassArgs a) {
    using T = typename S::Type;
    constexpr int DP = S::DP, NT = S::NT, MT = S::MT, KT = S::KT, NQ = S::NQ, kStages = S::kStages, kAhead = S::kAhead;
    constexpr int kVec = KvType<T>::kVec, kPieces = DP / kVec;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t s_row[2][KT];
    __shared__ __align__(16) float s_lse[NQ];
    __shared__ uint32_t s_anc[NQ];
    __shared__ int s_to[32];  // places of the pass's rows behind the kept ones
    __shared__ AttnCut s_cut;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int quad = lane >> 2, two = (lane & 3) * 2;
    const KvView& kv = a.kv;
    const uint32_t base_s = smem_u32(smem), sq = base_s + kStages * S::kTile;
    const int group = static_cast<int>(a.group.d), m_rows = a.rows * group;
    const float c_scale = attn_scale(a.scale);
    const int skip_blocks = a.skip / kv.block_size();

    AttnCursor cur, ahead, ids;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what the kernels before wrote
    const AttnRun run = attn_cut<S::kThreads, 0>(a, s_cut, KT, kv.heads, blockIdx.x, gridDim.x, cur);
    const int n = run.n;
    if (n == 0) return;
    ids = ahead = cur;

    // block numbers and copies run ahead of the products as in tree_attention_kernel
    struct Place {
        int blk, in, h;
    };
    int ids_i = 0;
    auto fetch_row = [&]() {
        Place p = {0, -1, 0};
        if (ids_i < n) {
            const int t = ids.tile * KT + tid;
            if (tid < KT && t < ids.len) {
                const int lb = kv.block.div(t);
                p.blk = kv.tables[static_cast<int64_t>(ids.b) * kv.max_blocks + skip_blocks + lb];
                p.in = t - lb * kv.block_size();
                p.h = ids.s;
            }
            ids.next(a, KT);
        }
        ++ids_i;
        return p;
    };
    auto post_row = [&](int i, const Place& p) {
        if (tid < KT) s_row[i & 1][tid] = p.in >= 0 && kv.valid(p.blk) ? kv.at(p.blk, p.h, p.in) : -1;
    };
    auto copy_tile = [&](int i) {
        if (i < n) {
            const uint32_t st = base_s + (i % kStages) * S::kTile;
            const T* k = static_cast<const T*>(kv.k);
            const int c = tid % kPieces;
            constexpr int kStep = S::kThreads / kPieces;
#pragma unroll
            for (int r = tid / kPieces; r < KT; r += kStep) {
                const int64_t at = s_row[i & 1][r];
                const bool take = at >= 0 && c * kVec < kv.dim;
                cp_async16(st + attn_at<S>(r, c), k + (take ? at + c * kVec : 0), take);
            }
            ahead.next(a, KT);
        }
        cp_commit();
    };
    // queries m0 .. m0 + NQ of kv head h: rows behind the last are zeros that take no part
    auto copy_queries = [&](int b, int h, int m0) {
        const T* q = static_cast<const T*>(a.q);
        const int c = tid % kPieces;
        for (int m = tid / kPieces; m < NQ; m += S::kThreads / kPieces) {
            const int row = m0 + m;
            const bool take = row < m_rows && c * kVec < kv.dim;
            const int r = a.group.div(row), g = row - r * group;
            const int64_t off = (static_cast<int64_t>(b) * a.rows + r) * a.q_stride +
                                (static_cast<int64_t>(h) * group + g) * kv.dim + c * kVec;
            cp_async16(sq + attn_at<S>(m, c), q + (take ? off : 0), take);
        }
    };
    // ... their sums (an infinite one: the row takes no part) and ancestors, by the whole CTA
    auto note_queries = [&](int b, int h, int m0, uint32_t line, uint32_t kept) {
        for (int m = tid; m < (NQ + 31) / 32 * 32; m += S::kThreads) {  // (whole warps: they shuffle)
            const int row = m0 + m;
            const bool real = row < m_rows;
            const int r = a.group.div(real ? row : 0), g = row - r * group;
            const uint32_t anc = __shfl_sync(0xffffffffu, line, r);
            if (m >= NQ) continue;
            float l = INFINITY;
            if (real && (kept >> r & 1))
                l = a.lse[(static_cast<int64_t>(b) * a.rows + r) * a.q_heads + static_cast<int64_t>(h) * group + g];
            s_lse[m] = fabsf(l) == INFINITY ? INFINITY : l * 1.44269504f;
            s_anc[m] = real ? anc : 0;
        }
    };

    Place places[kAhead + 1];
#pragma unroll
    for (int i = 0; i <= kAhead; ++i) places[i] = fetch_row();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        post_row(i, places[i]);
        __syncthreads();
        copy_tile(i);
    }
    Place place = places[kAhead];

    uint32_t line = 0, kept = ~0u;  // ancestors of row `lane`; the rows that take part
    bool refused = false;
    for (int i = 0; i < n; ++i) {
        post_row(i + kAhead, place);
        place = fetch_row();
        const bool starts = cur.tile == 0 || i == 0;
        if (starts) {  // a segment: its sequence's checks, alike in every CTA that has some of it
            int status = cur.len < 0 ? KV_LENGTH : 0;
            bool hole = false;
            int to = lane;
            if (cur.len > 0) {
                int depth;
                if (!warp_tree(a.parents ? a.parents + static_cast<int64_t>(cur.b) * (a.rows - 1) : nullptr, a.rows, lane,
                               line, depth))
                    status |= KV_PARENT;
                kept = mass_kept(a, cur.b, lane, to, status);
                const int32_t* table = kv.tables + static_cast<int64_t>(cur.b) * kv.max_blocks + skip_blocks;
                for (int x = tid, last = kv.block.div(cur.len - 1); x <= last; x += S::kThreads) hole |= !kv.valid(table[x]);
            }
            if (__syncthreads_or(hole)) status |= KV_BLOCK;
            if (warp == 0) s_to[lane] = to;  // (the last tile has read its own, before this barrier)
            refused = status != 0;
            if (tid == 0 && cur.tile == 0 && cur.s == 0 && a.row_status) a.row_status[cur.b] = status;
            if (cur.len > 0 && !refused) {
                copy_queries(cur.b, cur.s, 0);
                note_queries(cur.b, cur.s, 0, line, kept);
            }
            cp_commit();
            cp_wait<0>();
        } else {
            cp_wait<kAhead - 1>();
        }
        __syncthreads();
        copy_tile(i + kAhead);
        const uint32_t sk = base_s + (i % kStages) * S::kTile;
        const int t0 = cur.tile * KT + a.skip;           // of the sequence
        const int len = cur.len + a.skip, base = len - a.rows;
        if (cur.len > 0 && !refused) {
            const int pos0 = t0 + warp * 16 * MT + quad;  // of the thread's first position
            const int64_t line0 = (static_cast<int64_t>(cur.b) * kv.heads + cur.s) * a.width;
            float before[MT][2], sum[MT][2];
#pragma unroll
            for (int g = 0; g < MT; ++g)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int pos = pos0 + g * 16 + 8 * e;
                    before[g][e] = a.mass && (lane & 3) == 0 && pos >= a.first && pos < base ? a.mass[line0 + pos] : 0.0f;
                    sum[g][e] = 0.0f;
                }
            const bool edge = t0 + KT > base;
            for (int m0 = 0; m0 < m_rows; m0 += NQ) {
                if (m_rows > NQ && !(starts && m0 == 0)) {
                    // more queries than are kept: the next ones, for this tile
                    __syncthreads();
                    copy_queries(cur.b, cur.s, m0);
                    note_queries(cur.b, cur.s, m0, line, kept);
                    cp_commit();
                    cp_wait<0>();
                    __syncthreads();
                }
                float s[MT][NT][4];
#pragma unroll
                for (int g = 0; g < MT; ++g)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[g][t][e] = 0.0f;
                if constexpr (S::kBf16) {
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk) {
                        uint32_t kf[MT][4];
#pragma unroll
                        for (int g = 0; g < MT; ++g)
                            ldsm4(sk + attn_at<S>((warp * MT + g) * 16 + (lane & 15), kk * 2 + (lane >> 4)), kf[g]);
#pragma unroll
                        for (int t = 0; t < NT; t += 2) {
                            uint32_t qf[4];
                            ldsm4(sq + attn_at<S>((t * 8 + (lane & 7) + ((lane >> 4) << 3)) % NQ, kk * 2 + ((lane >> 3) & 1)),
                                  qf);
#pragma unroll
                            for (int g = 0; g < MT; ++g) {
                                mma_bf16(s[g][t], kf[g], qf[0], qf[1]);
                                if (t + 1 < NT) mma_bf16(s[g][t + 1 < NT ? t + 1 : t], kf[g], qf[2], qf[3]);
                            }
                        }
                    }
                } else {
                    // two tf32 parts each, as tree attention has them; the small products add up by themselves
                    float low[MT][NT][4] = {};
#pragma unroll 2
                    for (int kk = 0; kk < DP / 8; ++kk) {
                        uint32_t ah[MT][4], al[MT][4];
#pragma unroll
                        for (int g = 0; g < MT; ++g)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                split_tf32(ld_shared_f32(sk + attn_at<S>((warp * MT + g) * 16 + quad + 8 * (e & 1),
                                                                         kk * 2 + (e >> 1)) +
                                                         (lane & 3) * 4),
                                           ah[g][e], al[g][e]);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            uint32_t bh[2], bl[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                split_tf32(ld_shared_f32(sq + attn_at<S>(t * 8 + quad, kk * 2 + e) + (lane & 3) * 4), bh[e],
                                           bl[e]);
#pragma unroll
                            for (int g = 0; g < MT; ++g) {
                                mma_tf32(low[g][t], al[g], bh[0], bh[1]);
                                mma_tf32(low[g][t], ah[g], bl[0], bl[1]);
                                mma_tf32(s[g][t], ah[g], bh[0], bh[1]);
                            }
                        }
                    }
#pragma unroll
                    for (int g = 0; g < MT; ++g)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                s[g][t][e] += low[g][t][e];
                                // infinities and values near the ends of the type, as in tree attention
                                if (!finite(s[g][t][e]))
                                    s[g][t][e] = attn_dot<S>(sq, t * 8 + two + (e & 1), sk,
                                                             (warp * MT + g) * 16 + quad + 8 * (e >> 1));
                            }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if (m0 + t * 8 >= m_rows) break;
                    const float2 l = *reinterpret_cast<const float2*>(&s_lse[t * 8 + two]);
#pragma unroll
                    for (int g = 0; g < MT; ++g)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float m = e & 1 ? l.y : l.x;
                            // (a row that takes no part: not by its weight, as a score of infinity has none)
                            bool in = m != INFINITY;
                            if (edge) {
                                const int node = pos0 + g * 16 + 8 * (e >> 1) - base;
                                in = in && (node < 0 || (node < 32 && (s_anc[t * 8 + two + (e & 1)] >> node & 1)));
                            }
                            const float w = ex2(fmaf(s[g][t][e], c_scale, -m));
                            sum[g][e >> 1] += in ? w : 0.0f;
                        }
                }
            }
#pragma unroll
            for (int g = 0; g < MT; ++g)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    sum[g][e] += __shfl_xor_sync(0xffffffffu, sum[g][e], 1);
                    sum[g][e] += __shfl_xor_sync(0xffffffffu, sum[g][e], 2);
                    const int pos = pos0 + g * 16 + 8 * e;
                    // (a kept node moves to its place, maybe to one before `first`, which stays as it was)
                    const int to = pos >= base && pos < len ? s_to[pos - base] : 0;
                    const int at = pos >= base ? base + to : pos;
                    if ((lane & 3) == 0 && at >= a.first && pos < len && to >= 0)
                        a.out[line0 + at] = before[g][e] + sum[g][e];
                }
        }
        cur.next(a, KT);
    }
}

}  // namespace specv
