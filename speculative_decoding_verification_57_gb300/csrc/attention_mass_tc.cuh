// attention_mass_tc.cuh -- gathered attention weight in bf16 on the tcgen05
// tensor cores: head_dim up to 128, up to 256 queries a kv head.  Mathematics
// and work line as in attention_mass.cuh; a tile is 128 positions.
//
// The keys are the left operand: a position is a row of the scores, a lane of
// tensor memory, and a thread adds up the weights of its position over all
// queries by itself, with no exchange.  One CTA an SM: two groups of four
// warps take the tiles in turn, each with scores of its own in tensor memory;
// one warp issues the products, one brings the queries, their sums and trees
// a segment ahead (two sets, where 128 rows hold them), the others bring keys
// (boxes, or 16-byte copies, as tree_attention_tc.cuh has them).
//
// A position's row is told from others' at its store, so that keys behind a
// sequence's end need no care; columns without a query, rows whose lse is
// infinite and, near the pass's rows, hidden columns are left out by
// selection, where there are any.
//
// Measured (GB300, graph replays over sets of inputs beyond the L2; 32/8 heads of
// 128): single rows of 64 sequences over 1000..2000 positions 40.2 us, 75% of 6803
// GB/s, trees of 17 rows over 2048..4096 77.5 us, 79% (on mma.sync, whose scores
// have positions and queries in the same thread, 48 and 276).  Bound by memory:
// without loads 29 and 66 us, with an eighth of the weights 40 and 76.  Blocks are
// checked a segment ahead by the warp that brings the queries: by the weights' warps
// at a segment's start, single rows took 46 us.
#pragma once
#include "attention_mass.cuh"
#include "tree_attention_tc.cuh"

namespace specv {

template <int DP_, bool TMA_>
struct MassTc {
    static constexpr int DP = DP_;
    static constexpr bool TMA = TMA_;
    static constexpr int KT = 128;
    static constexpr int kPanel = 128 * 128;
    static constexpr int kPanels = DP / 64;
    static constexpr int kSlot = kPanels * kPanel;
    static constexpr int kSlots = DP == 64 ? 8 : 4;
    static constexpr int kRows = 256;  // queries, or two sets of 128
    static constexpr int kBoxWarps = 3;
    static constexpr int kThreads = 14 * 32;  // 8 for weights, products, queries, 4 for copies
};

template <typename S>
struct MassShared {
    unsigned char q[S::kRows * S::DP * 2];
    unsigned char slot[S::kSlots][S::kSlot];
    float lse[S::kRows];           // minus the sums, in base 2
    uint32_t anc[S::kRows];
    uint32_t part[S::kRows / 32];  // bit e of word c: row 32 c + e takes part
    AttnCut cut;
    uint64_t full[S::kSlots], empty[S::kSlots], q_full[2], q_empty[2], s_full[2], s_empty[2], end;
    int status[2];  // of a set's sequence
    int to[2][32];  // places of its pass's rows behind the kept ones
    int issued[S::kSlots];  // the last tile whose box was asked for
    uint32_t tmem;
    int fail;
};

// Where a run's segments and tiles are, for each role.
struct MassRun {
    AttnCursor cur;
    int left;  // tiles from the cursor on

    __device__ __forceinline__ int part() const { return tc_part(cur, left); }
    __device__ __forceinline__ void skip(const MassArgs& a, int nt) {
        left -= nt;
        cur.tile += nt - 1;
        cur.next(a, 128);
    }
};

// Queries, sums and ancestors of each segment, by one warp; and the statuses of the sequences that start in the run, of all
// of them, also behind a wait that ran out (which is told for them here and, as for the others, at the kernel's end).
template <typename S>
__device__ void mass_query_role(const MassArgs& a, MassShared<S>& sh, MassRun run, int sets, int lane) {
    const KvView& kv = a.kv;
    const int group = static_cast<int>(a.group.d), m_rows = a.rows * group, q_rows = S::kRows / sets;
    const int first_block = a.skip / kv.block_size();
    constexpr int kPieces = S::DP / 8;
    int checked = -1;
    bool holes = false, fine = true;  // no wait ran out; the same in all lanes
    for (int seg = 0; run.left > 0; ++seg) {
        const int set = sets == 2 ? seg & 1 : 0, turn = sets == 2 ? seg >> 1 : seg;
        const bool go = fine && (turn == 0 || tc_wait(smem_u32(&sh.q_empty[set]), (turn - 1) & 1, &sh.fail, a.polls));
        fine = __all_sync(0xffffffffu, go);
        const AttnCursor& cur = run.cur;
        if (!fine) {
            if (lane == 0 && cur.tile == 0 && cur.s == 0 && a.row_status) a.row_status[cur.b] = KV_TIMEOUT;
            run.skip(a, run.part());
            continue;
        }
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
        const uint32_t dst = smem_u32(sh.q) + set * q_rows * S::DP * 2;
        const int c = lane % kPieces;
        const bool col = c * 8 < kv.dim;
#pragma unroll 4
        for (int m = lane / kPieces; m < m_rows; m += 32 / kPieces) {
            const int r = a.group.div(m), g = m - r * group;
            const int64_t off = (static_cast<int64_t>(cur.b) * a.rows + r) * a.q_stride +
                                (static_cast<int64_t>(cur.s) * group + g) * kv.dim + c * 8;
            cp_async16(dst + (c >> 3) * q_rows * 128 + m * 128 + (((c & 7) ^ (m & 7)) << 4), q + (col ? off : 0), col);
        }
        uint32_t line;
        int depth;
        const bool ok = warp_tree(a.parents ? a.parents + static_cast<int64_t>(cur.b) * (a.rows - 1) : nullptr, a.rows, lane,
                                  line, depth);
        int to, path_status = 0;
        const uint32_t kept = mass_kept(a, cur.b, lane, to, path_status);
        sh.to[set][lane] = to;
        for (int m0 = 0; m0 < m_rows; m0 += 32) {
            const int m = m0 + lane, r = a.group.div(m < m_rows ? m : 0), g = m - r * group;
            const uint32_t anc = __shfl_sync(0xffffffffu, line, r);
            float l = INFINITY;
            if (m < m_rows && (kept >> r & 1))
                l = a.lse[(static_cast<int64_t>(cur.b) * a.rows + r) * a.q_heads + static_cast<int64_t>(cur.s) * group + g];
            const uint32_t part = __ballot_sync(0xffffffffu, fabsf(l) != INFINITY);
            if (lane == 0) sh.part[(set * q_rows + m0) >> 5] = part;
            sh.lse[set * q_rows + m] = l * -1.44269504f;
            sh.anc[set * q_rows + m] = anc;
        }
        // the sequence's blocks, all of them in every CTA that has some of it, once for all heads: of a refused sequence
        // nothing is written
        if (cur.b != checked) {
            bool hole = false;
            if (cur.len > 0) {
                const int32_t* table = kv.tables + static_cast<int64_t>(cur.b) * kv.max_blocks + first_block;
                const int last = kv.block.div(cur.len - 1);
#pragma unroll 16
                for (int i = lane; i <= last; i += 32) hole |= !kv.valid(table[i]);
            }
            holes = __any_sync(0xffffffffu, hole);
            checked = cur.b;
        }
        if (lane == 0) {
            const int status = cur.len < 0    ? KV_LENGTH
                               : cur.len == 0 ? 0
                                              : (ok ? 0 : KV_PARENT) | (holes ? KV_BLOCK : 0) | path_status;
            sh.status[set] = status;
            if (cur.tile == 0 && cur.s == 0 && a.row_status) a.row_status[cur.b] = status;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&sh.q_full[set]));
        run.skip(a, run.part());
    }
}

// Boxes: a tile a warp in turn, as tc_box_role brings them.  None is in flight when the CTA ends: the products waited for
// every tile, or a wait ran out, and then mass_boxes_land does.
template <typename S>
__device__ void mass_box_role(const MassArgs& a, const TcMaps& maps, MassShared<S>& sh, MassRun run, int warp,
                              int lane) {
    const KvView& kv = a.kv;
    const int panels = maps.flat ? 1 : S::kPanels, part = lane / panels, panel = lane % panels, rows = maps.rows;
    const bool mine = part * rows < S::KT;
    const int first_block = a.skip / kv.block_size(), n = run.left;
    const int withhold = blockIdx.x == 0 ? a.withhold : -1;
    for (int j = 0; j < n; ++j, run.cur.next(a, S::KT)) {
        if (j % S::kBoxWarps != warp) continue;
        const AttnCursor& cur = run.cur;
        const int t = cur.tile * S::KT + part * rows;
        const bool in = mine && t < cur.len;
        const int lb = kv.block.div(in ? t : 0);
        const int blk = in ? kv.tables[static_cast<int64_t>(cur.b) * kv.max_blocks + first_block + lb] : -1;
        const bool valid = kv.valid(blk);
        const int row = valid ? t - lb * kv.block_size() : 0;
        const int slot = j % S::kSlots;
        const bool go = j < S::kSlots || tc_wait(smem_u32(&sh.empty[slot]), (j / S::kSlots - 1) & 1, &sh.fail, a.polls);
        if (!__all_sync(0xffffffffu, go) || j == withhold) break;
        const uint32_t bar = smem_u32(&sh.full[slot]);
        if (lane == 0) {
            sh.issued[slot] = j;
            mbar_arrive_expect_tx(bar, S::kSlot);
        }
        __syncwarp();
        if (mine && maps.flat)
            tc_box2(smem_u32(sh.slot[slot]) + part * rows * 256, &maps.k, row >> 3,
                    (valid ? blk : kv.blocks) * maps.flat + (valid ? cur.s : 0), bar);
        else if (mine)
            tc_box(smem_u32(sh.slot[slot]) + panel * S::kPanel + part * rows * 128, &maps.k, panel * 64, row, cur.s,
                   valid ? blk : kv.blocks, bar);
    }
}

// Behind a wait that ran out, when every role is done: the last box of each slot has landed (what filled the slot before it was
// used up).  Only then do the phases stand still: a warp that looked back at its own boxes while another filled a slot again, and
// the products used that up, took the parities of both barriers for those of a box in flight and stood for its 200 ms, once in
// some 50,000 calls.
template <typename S>
__device__ __forceinline__ void mass_boxes_land(MassShared<S>& sh, int tid) {
    if (tid < S::kSlots && sh.issued[tid] >= 0)
        mbar_wait_bounded(smem_u32(&sh.full[tid]), (sh.issued[tid] / S::kSlots) & 1, 1u << 30);
}

// 16-byte copies by four warps; a tile is told when those of two tiles on are under way.
template <typename S>
__device__ void mass_copy_role(const MassArgs& a, MassShared<S>& sh, MassRun run, int p) {
    constexpr int kPieces = S::DP / 8, kStep = 128 / kPieces, kOwn = 32 / kPieces, kBehind = 2;
    const KvView& kv = a.kv;
    const int lane = p & 31, warp = p >> 5, c = p % kPieces, r0 = p / kPieces;
    const int mine = (lane / kOwn) * kStep + warp * kOwn + lane % kOwn;  // the row whose place this lane finds
    const bool col = c * 8 < kv.dim;
    const int first_block = a.skip / kv.block_size(), n = run.left;
    const int withhold = blockIdx.x == 0 ? a.withhold : -1;
    auto tell = [&](int j) {
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&sh.full[j % S::kSlots]));
    };
    int j = 0;
    for (; j < n; ++j, run.cur.next(a, S::KT)) {
        const AttnCursor& cur = run.cur;
        int64_t at = -1;
        const int t = cur.tile * S::KT + mine;
        if (t < cur.len) {
            const int lb = kv.block.div(t);
            const int blk = kv.tables[static_cast<int64_t>(cur.b) * kv.max_blocks + first_block + lb];
            if (kv.valid(blk)) at = kv.at(blk, cur.s, t - lb * kv.block_size());
        }
        const int slot = j % S::kSlots;
        const bool go = j < S::kSlots || tc_wait(smem_u32(&sh.empty[slot]), (j / S::kSlots - 1) & 1, &sh.fail, a.polls);
        if (!__all_sync(0xffffffffu, go) || j == withhold) break;
        const uint32_t dst = smem_u32(sh.slot[slot]);
#pragma unroll
        for (int i = 0; i < S::KT / kStep; ++i) {
            const int64_t from = __shfl_sync(0xffffffffu, at, i * kOwn + lane / kPieces);
            const bool take = from >= 0 && col;
            const int r = r0 + i * kStep;
            cp_async16(dst + (c >> 3) * S::kPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                       static_cast<const __nv_bfloat16*>(kv.k) + (take ? from + c * 8 : 0), take);
        }
        cp_commit();
        if (j >= kBehind) {
            cp_wait<kBehind>();
            tell(j - kBehind);
        }
    }
    cp_wait<0>();
    for (int i = j > kBehind ? j - kBehind : 0; i < j; ++i) tell(i);
}

// Products: 128 positions by the queries, one warp.
template <typename S>
__device__ void mass_mma_role(const MassArgs& a, MassShared<S>& sh, const TcLayout& lay, MassRun run, int sets) {
    const int m_rows = a.rows * static_cast<int>(a.group.d), q_rows = S::kRows / sets;
    const uint32_t idesc = tc_idesc((m_rows + 15) / 16 * 16, false);
    const uint32_t tm = __shfl_sync(0xffffffffu, sh.tmem, 0);
    bool fine = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        fine = __all_sync(0xffffffffu, fine && tc_wait(smem_u32(bar), parity, &sh.fail, a.polls));
    };
    int j = 0;
    for (int seg = 0; fine && run.left > 0; ++seg) {
        const int set = sets == 2 ? seg & 1 : 0, turn = sets == 2 ? seg >> 1 : seg, nt = run.part();
        wait(&sh.q_full[set], turn & 1);
        const uint64_t qd = tc_desc_rows(smem_u32(sh.q) + set * q_rows * S::DP * 2, 1024);
        for (int t = 0; fine && t < nt; ++t, ++j) {
            const int slot = __shfl_sync(0xffffffffu, j % S::kSlots, 0), x = j & 1;
            wait(&sh.full[slot], (j / S::kSlots) & 1);
            if (j >= 2) wait(&sh.s_empty[x], ((j >> 1) - 1) & 1);
            if (!fine) break;
            tc_after_sync();
            if (tc_elect()) {
                const uint64_t kd = tc_desc_rows(smem_u32(sh.slot[slot]), lay.step);
#pragma unroll
                for (int kk = 0; kk < S::DP / 16; ++kk)
                    tc_mma_ss(tm + x * 256, kd + (((kk >> 2) * lay.panel + (kk & 3) * 32) >> 4),
                              qd + (((kk >> 2) * q_rows * 128 + (kk & 3) * 32) >> 4), idesc, kk > 0);
                tc_commit(smem_u32(&sh.s_full[x]));
                tc_commit(smem_u32(&sh.empty[slot]));
                if (t + 1 == nt) tc_commit(smem_u32(&sh.q_empty[set]));
            }
            __syncwarp();
        }
        run.skip(a, nt);
    }
    // nothing of this warp's is in flight when tensor memory is freed
    if (tc_elect()) tc_commit(smem_u32(&sh.end));
    __syncwarp();
    mbar_wait_bounded(smem_u32(&sh.end), 0, 1u << 30);
}

// Weights of a position over 32 queries, of those whose bit is set in `keep`;
// eight that nobody in the warp keeps are passed over.
template <bool SELECT>
__device__ __forceinline__ f2 mass_weights(const uint32_t (&s)[32], const float* lse, uint32_t keep, float scale, f2 sum) {
    const f2 sc = pack2(scale, scale);
    f2 other = pack2(0.0f, 0.0f);
#pragma unroll
    for (int e0 = 0; e0 < 32; e0 += 8) {
        if (SELECT && !__any_sync(0xffffffffu, keep >> e0 & 0xff)) continue;
#pragma unroll
        for (int e = e0; e < e0 + 8; e += 4) {
            const float4 l = *reinterpret_cast<const float4*>(lse + e);
            float w[4];
            unpack2(fma2(pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc, pack2(l.x, l.y)), w[0], w[1]);
            unpack2(fma2(pack2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), sc, pack2(l.z, l.w)), w[2], w[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = ex2(w[k]);
                if (SELECT) w[k] = keep >> (e + k) & 1 ? w[k] : 0.0f;
            }
            sum = add2(sum, pack2(w[0], w[1]));
            other = add2(other, pack2(w[2], w[3]));
        }
    }
    return add2(sum, other);
}

// Weights, of every second tile: four warps, a thread a position.
template <typename S>
__device__ void mass_weight_role(const MassArgs& a, MassShared<S>& sh, MassRun run, int sets, int x, int row) {
    const KvView& kv = a.kv;
    const int lane = row & 31, m_rows = a.rows * static_cast<int>(a.group.d), q_rows = S::kRows / sets;
    const uint32_t ts = sh.tmem + x * 256 + (static_cast<uint32_t>(row & ~31) << 16);
    const float scale = attn_scale(a.scale);
    bool fine = true;  // the same in all lanes
    int j = 0;
    for (int seg = 0; run.left > 0; ++seg) {
        const int set = sets == 2 ? seg & 1 : 0, turn = sets == 2 ? seg >> 1 : seg, nt = run.part();
        const AttnCursor cur = run.cur;
        fine = fine && tc_wait(smem_u32(&sh.q_full[set]), turn & 1, &sh.fail, a.polls);
        fine = __all_sync(0xffffffffu, fine);
        const int status = sh.status[set];
        const float* lse = sh.lse + set * q_rows;
        const uint32_t* anc = sh.anc + set * q_rows;
        const int len = cur.len + a.skip, base = len - a.rows;
        const int64_t line0 = (static_cast<int64_t>(cur.b) * kv.heads + cur.s) * a.width;
        for (int t = 0; t < nt; ++t, ++j) {
            if ((j & 1) != x || !fine) continue;
            const int t0 = (cur.tile + t) * S::KT + a.skip, pos = t0 + row;
            const bool writes = cur.len > 0 && status == 0 && pos >= a.first && pos < len;
            const float before = writes && a.mass && pos < base ? a.mass[line0 + pos] : 0.0f;
            fine = __all_sync(0xffffffffu, tc_wait(smem_u32(&sh.s_full[x]), (j >> 1) & 1, &sh.fail, a.polls));
            if (!fine) continue;
            tc_after_sync();
            const bool edge = t0 + S::KT > base;
            const int node = pos - base;
            f2 sum = pack2(0.0f, 0.0f);
            for (int c = 0; c < m_rows; c += 32) {
                uint32_t s[32];
                tc_ld32(ts + c, s);
                tc_wait_ld();
                if (c + 32 >= m_rows) {  // the scores are read
                    tc_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.s_empty[x]));
                }
                uint32_t keep = sh.part[(set * q_rows + c) >> 5];
                if (edge) {  // of the pass's rows a position is seen by its own and those below
                    uint32_t seen = 0;
#pragma unroll
                    for (int e = 0; e < 32; ++e) seen |= (anc[c + e] >> (node & 31) & 1) << e;
                    if (node >= 0) keep &= seen;
                }
                if (__all_sync(0xffffffffu, keep == ~0u))
                    sum = mass_weights<false>(s, lse + c, keep, scale, sum);
                else
                    sum = mass_weights<true>(s, lse + c, keep, scale, sum);
            }
            float lo, hi;
            unpack2(sum, lo, hi);
            // (a kept node moves to its place, maybe to one before `first`, which stays as it was)
            const int to = node >= 0 && node < 32 ? sh.to[set][node] : 0, at = node >= 0 ? base + to : pos;
            if (writes && to >= 0 && at >= a.first) a.out[line0 + at] = before + (lo + hi);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.q_empty[set]));
        run.skip(a, nt);
    }
}

template <typename S>
__global__ void __launch_bounds__(S::kThreads, 1)
attention_mass_tc_kernel(const MassArgs a, const __grid_constant__ TcMaps maps) {
    extern __shared__ __align__(1024) unsigned char tc_smem[];
    MassShared<S>& sh = *reinterpret_cast<MassShared<S>*>(tc_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if constexpr (S::TMA) {
        if (tid == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.k) : "memory");
    }
    MassRun run;
    run.cur.b = 0;
    attn_wait();
    const AttnRun cut = attn_cut<S::kThreads, 0>(a, sh.cut, S::KT, a.kv.heads, blockIdx.x, gridDim.x, run.cur);
    run.left = cut.n;
    if (cut.n == 0) return;
    const int sets = a.rows * static_cast<int>(a.group.d) <= S::kRows / 2 ? 2 : 1;
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(smem_u32(&sh.full[i]), S::TMA ? 1 : 128);
            mbar_init(smem_u32(&sh.empty[i]), 1);
            sh.issued[i] = -1;
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&sh.q_full[x]), 32);
            mbar_init(smem_u32(&sh.q_empty[x]), 1 + 8);  // the products, the warps with weights
            mbar_init(smem_u32(&sh.s_full[x]), 1);
            mbar_init(smem_u32(&sh.s_empty[x]), 4);
        }
        mbar_init(smem_u32(&sh.end), 1);
        fence_mbar_init();
        sh.fail = (smem_u32(tc_smem) & 1023) != 0;
    }
    __syncwarp();
    if (warp == 8) tc_alloc(smem_u32(&sh.tmem), 512);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const int b0 = run.cur.b;
    if (warp < 8)
        mass_weight_role<S>(a, sh, run, sets, warp >> 2, tid & 127);
    else if (warp == 8)
        mass_mma_role<S>(a, sh, tc_layout<S>(maps), run, sets);
    else if (warp == 9)
        mass_query_role<S>(a, sh, run, sets, lane);
    else if constexpr (S::TMA) {
        if (warp < 10 + S::kBoxWarps) mass_box_role<S>(a, maps, sh, run, warp - 10, lane);
    } else {
        mass_copy_role<S>(a, sh, run, tid - 320);
    }
    __syncwarp();
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == 8) tc_dealloc(sh.tmem, 512);
    if (S::TMA && tc_failed(&sh.fail)) {
        mass_boxes_land(sh, tid);
        __syncthreads();
    }
    // a wait that ran out, after all others are long done, is told for every sequence that the run touches
    if (tid == 0 && tc_failed(&sh.fail) && a.row_status) {
        for (int left = run.left; left > 0;) {
            const int nt = tc_part(run.cur, left);
            left -= nt;
            run.cur.tile += nt - 1;
            if (left > 0) run.cur.next(a, S::KT);
        }
        for (int b = b0; b <= run.cur.b; ++b) atomicOr(a.row_status + b, KV_TIMEOUT);
    }
}

}  // namespace specv
