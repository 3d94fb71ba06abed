// tree_attention_tc.cuh -- tree attention in bf16 on the tcgen05 tensor cores,
// head_dim up to 128.  Mathematics, work line and joining as in
// tree_attention.cuh; a tile is 128 positions, a row tile 128 rows.
//
// One CTA an SM, 12 or 16 warps: two streams of four softmax warps, two warps
// that issue the products, and those that bring keys and values: two or three
// for boxes, four that copy.  Registers move to the softmax warps.  A stream
// has the scores of one row tile and tile of positions (128 x 128 fp32) and
// its outputs (128 x DP fp32) in tensor memory; a softmax thread owns a row,
// so that maxima and sums need no exchange.  While one stream's weights are
// formed the tensor cores work on the other's products.  With up to 128 rows a kv head the streams take
// tiles of positions in turn and their outputs join at the segment's end;
// with more (WIDE) each has a row tile of its own and both use every tile.
//
// Weights go back to tensor memory over the scores they came from, in bf16,
// as the left operand of the product with the values; keys lie in shared
// memory with head_dim along the contraction, values with the positions along
// it, both as they lie in the cache, in 128-byte swizzled panels of 64
// columns.
//
// Blocks whose rows fill tiles evenly (a multiple of eight that divides 128,
// or a multiple of 128) come as tensor boxes, a box a block (of heads of 128) or
// a block and panel; others by 16-byte copies.  Boxes land where the tensor cores
// see them at once and cost the softmax warps' schedulers next to nothing (with
// the issuing warps' turns, they took the trees and the wide trees of the list
// below from 178 and 149 us to 156 and 129).
//
// Measured (GB300, 2070 MHz, graph replays over sets of inputs of more than
// twice the L2; bytes and operations counted once; of 6803 GB/s and 1896 TFLOP/s measured):
//   64 chains of 6 rows, 32/8 heads of 128, 1000..2000 positions    77 us  76%
//   64 trees of 17 rows, same heads, 2048..4096                    144 us  85%
//   one tree of 17 rows, same heads, 131072                         94 us  84%
//   16 trees of 32 rows, 64/8 heads, 4096..8192 (WIDE)             103 us  61%,
//     1015 TFLOP/s, 54%
// With one row tile the memory bounds it, short of it by each run's start
// (5 us), its segments' ends and the join (5 to 10 us).  WIDE, two streams take
// 3050 cycles for a tile each, 2048 of them for their 32 products: a stream has
// its scores, 1050 cycles on the first half of its weights are ready, 550 later
// the second, 1400 on from the first half its next scores.  Halving the
// products' columns gains 3%, the maxima left out 3%, a second of the parts no
// more: the hand-overs bound it, four of some 150 cycles.  Not built, as they
// gained nothing here: maxima formed beside the first half's weights (spills: 199 us
// for 175 with the trees behind a prefix), one issuing warp for both streams (203),
// waits that poll without rest (268).
#pragma once
#include <cuda.h>

#include "tree_attention.cuh"

namespace specv {

// ------------------------------------------------------------------ tcgen05
__device__ __forceinline__ void tc_alloc(uint32_t smem_dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane of a converged warp, the same every time.  Products are issued in
// branches on this: told by a lane's number instead, the compiler cannot see
// that one thread runs them, and an instruction took 80 to 100 cycles to
// issue, more than its 64 on the tensor cores (64 trees of 17 rows behind a
// prefix of 8192 positions: 216 us for 204).
__device__ __forceinline__ bool tc_elect() {
    uint32_t x;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(x));
    return x != 0;
}

// Arrives on `bar` when every product that this thread issued so far is done.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// d (+)= a b, a and b in shared memory
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// d (+)= a b, a in tensor memory
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// 32 columns of the warp's 32 lanes, a lane a thread
__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
            r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}

// Shared memory operands in 128-byte swizzled panels (64 columns of bf16; row
// r at 128 r, eight rows an atom of 1024 bytes).
// ... contraction along the columns: atoms `step` bytes apart along the rows
__device__ __forceinline__ uint64_t tc_desc_rows(uint32_t addr, uint32_t step) {
    return (2ull << 61) | (1ull << 46) | (static_cast<uint64_t>(step >> 4) << 32) | (1ull << 16) | ((addr >> 4) & 0x3fff);
}
// ... contraction along the rows: atoms `step` bytes apart along it, panels `panel` bytes apart along the columns
__device__ __forceinline__ uint64_t tc_desc_cols(uint32_t addr, uint32_t step, uint32_t panel) {
    return (2ull << 61) | (1ull << 46) | (static_cast<uint64_t>(step >> 4) << 32) |
           (static_cast<uint64_t>(panel >> 4) << 16) | ((addr >> 4) & 0x3fff);
}

// bf16 x bf16 -> fp32, 128 rows, n columns; cols: the right operand's contraction runs along its rows
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool cols) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (cols ? 1u << 16 : 0u) | (static_cast<uint32_t>(n / 8) << 17) |
           (128u / 16 << 24);
}

// ------------------------------------------------------------------ shapes
template <int DP_, bool WIDE_, bool TMA_, int BOXES = 2>
struct TcShape {
    using Type = __nv_bfloat16;
    static constexpr int DP = DP_;
    static constexpr bool WIDE = WIDE_;
    static constexpr bool TMA = TMA_;  // blocks come as tensor boxes; else by 16-byte copies
    static constexpr int kTiles = WIDE ? 2 : 1;  // row tiles of a segment
    static constexpr int TM = 128 * kTiles;
    static constexpr int KT = 128;
    static constexpr int kPanel = 128 * 128;  // bytes of 128 rows of 64 columns
    static constexpr int kPanels = DP / 64;
    static constexpr int kSlot = kPanels * kPanel;  // keys, or values, of a tile
    static constexpr int kQ = kTiles * kSlot;
    // Slots for keys and values alike, filled and freed in the order of their
    // use: keys of a part's first kLead tiles, then values of tile t and keys
    // of tile t + kLead in turn.  160 to 192 KB: an SM's share of the memory's
    // rate times its latency several times over.
    static constexpr int kLead = WIDE ? 1 : 2;
    static constexpr int kSlots = DP == 64 ? 10 : WIDE ? 5 : 6;
    // Warps that bring boxes: two, or three for row tiles of 128 that the L2 serves at the tensor cores' pace (16 chains of
    // 6 rows behind 65536 positions 104 us with three, 119 with two), at the price of registers (in 12 warps trees of 32
    // rows with 64 heads take 104 us, in 16 107; chains of 6 rows over 2000 positions 78 and 82).
    static constexpr int kBoxWarps = BOXES;
    // of a segment, besides its tiles, in tiles (64 trees of 17 rows over 4096 positions: 0 152 us, 2 149, 4 147; 64 chains
    // of 6 over 2000: 80.5, 77.2, 76.7; WIDE, 16 trees of 32 rows with 64 heads over 8192: 0 114, 2 109.4, 3 109.2, 4 109.5)
    static constexpr int kCost = WIDE ? 3 : 4;
    // eight warps of softmax, two of products, and those for boxes, or four that copy and one that shows
    static constexpr bool kTwelve = TMA && BOXES == 2;
    static constexpr int kThreads = (kTwelve ? 12 : 16) * 32;
    // registers of a softmax thread, and of the others: together those that the launch has
    static constexpr int kMany = kTwelve ? 208 : 176, kFew = kTwelve ? 88 : 80;
    static_assert(256 * kMany + (kThreads - 256) * kFew <= kThreads * (65536 / kThreads / 8 * 8), "registers of the launch");
    // place, in the order of use from its part's first slot on, of the values of tile t of nt
    static __device__ __forceinline__ int values_at(int t, int nt) {
        const int more = nt > kLead ? nt - kLead : 0;
        return (nt < kLead ? nt : kLead) + t + (t < more ? t : more);
    }
    // ... and of its keys
    static __device__ __forceinline__ int keys_at(int t, int nt) {
        return t < kLead ? t : values_at(t - kLead, nt) + 1;
    }
};

// How the keys and values of a tile lie in their slot: eight rows of a panel
// are 1024 bytes; `step` bytes on lie the next eight rows, `panel` bytes on the
// next panel of the same rows.
struct TcLayout {
    uint32_t step, panel;

    __device__ __forceinline__ uint32_t at(int row, int piece) const {  // byte offset of 16-byte piece `piece` of a row
        return (piece >> 3) * panel + (row >> 3) * step + (row & 7) * 128 + (((piece & 7) ^ (row & 7)) << 4);
    }
};

// Tensor maps of the two pools ([blocks, heads, block_size, head_dim], boxes
// of `rows` rows of 64 columns), where boxes are used, and of the queries
// ([batch, rows, heads, head_dim], boxes of a group of heads of q_rows rows,
// 128 rows of a row tile) where groups fill row tiles (q_rows 0: they do not).
// Rows of 128 values in pools whose blocks lie whole heads apart come with both
// panels in one box ([blocks and heads, block_size / 8, 2, 8, 64]: `flat` heads
// from a block to the next; else 0): half as many boxes, of which a warp takes
// some 90 cycles each to issue.
struct TcMaps {
    CUtensorMap k, v, q;
    int rows, q_rows, flat;
};

template <typename S>
__device__ __forceinline__ TcLayout tc_layout(const TcMaps& maps) {
    return S::TMA && maps.flat ? TcLayout{2048, 1024} : TcLayout{1024, S::kPanel};
}

template <typename S>
struct TcShared {
    unsigned char q[S::kQ];
    unsigned char slot[S::kSlots][S::kSlot];
    float2 ml[S::WIDE ? 1 : 2][S::WIDE ? 1 : 128];  // the streams' maxima and sums, as they join
    AttnCut cut;
    // a slot's copies have landed, are visible to the tensor cores, are used up
    uint64_t full[S::kSlots], shown[S::kSlots], empty[S::kSlots];
    uint64_t q_full, q_shown, q_empty, s_full[2], p_half[2], p_ready[2], o_done[2], turn[2], end[2];
    uint32_t wild[16];  // by segment: nodes with values that are not finite ...
    int hole[16];       // ... and whether a block is outside the pool
    uint32_t tmem;
    int fail;          // a wait ran out: no role waits any more
    AttnCursor start;  // of the run
};

// A wait of a role: bounded, and none after one ran out.  False: it, or
// another, ran out; the role copies and issues nothing more.  A parity tells
// two successive phases apart and no more: who waits for a phase has to know
// that the one before it is complete.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t phase, int* fail, uint32_t polls) {
    if (mbar_test_wait(bar, phase)) return true;
    if (*static_cast<volatile int*>(fail)) return false;
    if (mbar_wait_bounded(bar, phase, polls)) return true;
    *static_cast<volatile int*>(fail) = 1;
    return false;
}
__device__ __forceinline__ bool tc_failed(const int* fail) { return *static_cast<const volatile int*>(fail) != 0; }

// Where a segment's part in a run ends: its tiles from cur.tile on, `left` tiles of the run to go.
__device__ __forceinline__ int tc_part(const AttnCursor& cur, int left) {
    return cur.tiles - cur.tile < left ? cur.tiles - cur.tile : left;
}

// The copies this thread issued so far arrive on `bar` when they have landed.
__device__ __forceinline__ void tc_copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A box of a block: 64 columns from `col` on of rows `row`.. of a head.
__device__ __forceinline__ void tc_box(uint32_t dst, const CUtensorMap* map, int col, int row, int h, int blk,
                                       uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(col), "r"(row), "r"(h), "r"(blk), "r"(bar)
        : "memory");
}

// Both panels of rows 8 `row8` .. of a head of a block.
__device__ __forceinline__ void tc_box2(uint32_t dst, const CUtensorMap* map, int row8, int head, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(0), "r"(row8), "r"(head), "r"(bar)
        : "memory");
}

// The slots of a run in the order of their use.
template <typename S>
struct TcUses {
    AttnCursor cur;  // at a part's first tile
    int n, nt;       // tiles from it on to the run's end, and of the part
    int u = 0, seg = 0;

    __device__ __forceinline__ TcUses(const AttnCursor& c, int n_) : cur(c), n(n_), nt(tc_part(c, n_)) {}
    template <typename A>
    __device__ __forceinline__ void next(const A& a) {
        if (++u < 2 * nt) return;
        u = 0;
        ++seg;
        n -= nt;
        cur.tile += nt - 1;
        cur.next(a, S::KT);
        nt = tc_part(cur, n);
    }
    // whether the use is of values, and its tile
    __device__ __forceinline__ bool what(int& tile) const {
        const int lead = nt < S::kLead ? nt : S::kLead, w = u - lead, pairs = 2 * (nt - lead);
        const bool values = w >= 0 && (w >= pairs || !(w & 1));
        tile = cur.tile + (w < 0 ? u : w >= pairs ? w - (nt - lead) : (w >> 1) + (w & 1 ? lead : 0));
        return values;
    }
};

// ------------------------------------------------------------------ copies
// Queries of a segment's row tiles, by THREADS threads (a multiple of a row's
// pieces apart), p of them this one.
template <typename S, int THREADS>
__device__ __forceinline__ void tc_copy_queries(const AttnArgs& a, TcShared<S>& sh, const AttnCursor& cur, int p) {
    using T = typename S::Type;
    constexpr int kPieces = S::DP / 8, kStep = THREADS / kPieces;
    const KvView& kv = a.kv;
    const int c = p % kPieces, h = cur.s / a.row_tiles, rt = cur.s - h * a.row_tiles;
    const int m_rows = a.rows * static_cast<int>(a.group.d);
    const T* q = static_cast<const T*>(a.q);
    // (rows behind the last keep what shared memory held: nobody reads their results)
    const int last = m_rows - rt * S::TM < S::TM ? m_rows - rt * S::TM : S::TM;
#pragma unroll 4
    for (int m = p / kPieces; m < last; m += kStep) {
        const int row = rt * S::TM + m;
        const bool take = c * 8 < kv.dim;
        const int r = a.group.div(row), g = row - r * static_cast<int>(a.group.d);
        const int64_t off = (static_cast<int64_t>(cur.b) * a.rows + r) * a.q_stride +
                            (static_cast<int64_t>(h) * a.group.d + g) * kv.dim + c * 8;
        cp_async16(smem_u32(sh.q) + (m >> 7) * S::kSlot + (c >> 3) * S::kPanel + (m & 127) * 128 + (((c & 7) ^ (m & 7)) << 4),
                   q + (take ? off : 0), take);
    }
}

// Boxes (TMA): kBoxWarps warps, a slot each in turn (a box takes a warp some 90
// cycles to issue, and a slot is up to 32 of them; sharing each slot's boxes
// instead was slower, 64 trees of 17 rows over 4096 positions 173 us for 160).  Lane l brings a panel of
// one of the tile's blocks; its block number is read a slot ahead.  A block
// that is outside the pool or past the sequence's end is asked for at block
// number `blocks`, which reads as zeros.
template <typename S, typename A>
__device__ void tc_box_role(const A& a, const TcMaps& maps, TcShared<S>& sh, const AttnCursor& cur, int n,
                            int warp, int lane) {
    const KvView& kv = a.kv;
    const int panels = maps.flat ? 1 : S::kPanels;
    const int part = lane / panels, panel = lane % panels;         // block of the tile, and columns
    const int rows = maps.rows;                                    // of a box
    const bool mine = part * rows < S::KT;
    const int first_block = attn_first_block(a);
    TcUses<S> it(cur, n);
    // what this lane asks for: block number (0: nothing to ask), and where in it
    struct Box {
        int blk, row, h, seg;
        bool values, in;
    };
    auto read = [&]() {
        Box x;
        int tile;
        x.values = it.what(tile);
        const int t = tile * S::KT + part * rows;
        x.in = mine && t < it.cur.len;
        const int lb = kv.block.div(x.in ? t : 0);
        x.blk = x.in ? kv.tables[static_cast<int64_t>(it.cur.b) * kv.max_blocks + first_block + lb] : 0;
        x.row = t - lb * kv.block_size();
        x.h = it.cur.s / a.row_tiles;
        x.seg = it.seg;
        return x;
    };
    // to use `to` of the run, from use `at`
    auto go = [&](int at, int to) {
        for (; at < to && at < 2 * n; ++at) {
            if (it.u == 0 && warp == 0 && lane == 0) {  // flags of a later segment; the roles are never that far apart
                sh.wild[(it.seg + 8) & 15] = 0;
                sh.hole[(it.seg + 8) & 15] = 0;
            }
            it.next(a);
        }
    };
    go(0, warp);
    const int withhold = blockIdx.x == 0 ? a.withhold : -1;
    Box next = {};
    if (warp < 2 * n) next = read();
    int use = warp;
    for (; use < 2 * n; use += S::kBoxWarps) {
        const Box x = next;
        go(use, use + S::kBoxWarps);
        if (use + S::kBoxWarps < 2 * n) next = read();
        const int slot = use % S::kSlots;
        // (whose phase before, kSlots uses earlier, this warp's last wait implies: slots are used up in order)
        bool go_on = use < S::kSlots || tc_wait(smem_u32(&sh.empty[slot]), (use / S::kSlots - 1) & 1, &sh.fail, a.polls);
        go_on = __all_sync(0xffffffffu, go_on);
        if (!go_on || use == withhold) break;
        const uint32_t bar = smem_u32(&sh.full[slot]);
        const bool valid = x.in && kv.valid(x.blk);
        if (x.in && !valid) sh.hole[x.seg & 15] = 1;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(bar, S::kSlot);
        __syncwarp();
        if (mine && maps.flat)
            tc_box2(smem_u32(sh.slot[slot]) + part * rows * 256, x.values ? &maps.v : &maps.k, valid ? x.row >> 3 : 0,
                    (valid ? x.blk : kv.blocks) * maps.flat + (valid ? x.h : 0), bar);
        else if (mine)
            tc_box(smem_u32(sh.slot[slot]) + panel * S::kPanel + part * rows * 128, x.values ? &maps.v : &maps.k,
                   panel * 64, valid ? x.row : 0, x.h, valid ? x.blk : kv.blocks, bar);
    }
    // no box of this warp's is in flight when the CTA ends, not even after a wait that ran out (those of kSlots uses
    // before the last and earlier had landed: their slots were used up).  Another warp may have filled a slot again since,
    // so that its parity is back where it was: then the slot had been used up, which its other barrier tells
    const int end = use;
    const unsigned long long since = gtimer();
    for (use = end - S::kBoxWarps; use >= 0 && use > end - S::kSlots; use -= S::kBoxWarps) {
        const uint32_t bar = smem_u32(&sh.full[use % S::kSlots]), used = smem_u32(&sh.empty[use % S::kSlots]);
        const uint32_t phase = (use / S::kSlots) & 1;
        while (!mbar_test_wait(used, phase) && !mbar_wait_bounded(bar, phase, 256) && gtimer() - since < kWaitNs) {
        }
    }
}

// Queries of a segment where the keys and values are boxes, by the warp that
// issues the first products with them: by boxes of their own or, where groups
// of heads do not fill row tiles, by 16-byte copies.
template <typename S, typename A>
__device__ __forceinline__ void tc_queries(const A& a, const TcMaps& maps, TcShared<S>& sh, const AttnCursor& cur, int p) {
    const uint32_t bar = smem_u32(&sh.q_shown);
    if (maps.q_rows) {
        // box p: panel p % kPanels of row tile p / kPanels; tiles behind the last row are left out
        const int h = cur.s / a.row_tiles, rt = cur.s - h * a.row_tiles;
        const int tile = p / S::kPanels, panel = p % S::kPanels;
        const int r = (rt * S::kTiles + tile) * maps.q_rows;
        const bool mine = tile < S::kTiles && r < a.rows;
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
        if (p == 0) mbar_arrive_expect_tx(bar, boxes * S::kPanel);
        __syncwarp();
        if (mine)
            tc_box(smem_u32(sh.q) + tile * S::kSlot + panel * S::kPanel, &maps.q, panel * 64,
                   h * static_cast<int>(a.group.d), r, cur.b, bar);
    } else {
        tc_copy_queries<S, 32>(a, sh, cur, p);
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        mbar_arrive(bar);
    }
    __syncwarp();
}

// 16-byte copies: four warps.  A warp copies 32 rows of every tile; lane l
// finds the place of one of them in the pool (while the slot it goes to is
// still in use) and hands it to the lanes that copy the row's pieces.
template <typename S, typename A>
__device__ void tc_copy_role(const A& a, TcShared<S>& sh, const AttnCursor& cur, int n, int p) {
    using T = typename S::Type;
    constexpr int kPieces = S::DP / 8;    // 16-byte pieces of a row
    constexpr int kStep = 128 / kPieces;  // rows a pass of the 128 threads
    constexpr int kOwn = 32 / kPieces;    // rows a pass of a warp
    const KvView& kv = a.kv;
    const int lane = p & 31, warp = p >> 5;
    const int c = p % kPieces, r0 = p / kPieces;
    const int mine = (lane / kOwn) * kStep + warp * kOwn + lane % kOwn;  // the row whose place this lane finds
    const bool col = c * 8 < kv.dim;
    const int withhold = blockIdx.x == 0 ? a.withhold : -1;
    const int first_block = attn_first_block(a);
    TcUses<S> it(cur, n);
    for (int use = 0; use < 2 * n; ++use, it.next(a)) {
        if (it.u == 0) {
            if (p == 0) {  // flags of a later segment; the roles are never that far apart
                sh.wild[(it.seg + 8) & 15] = 0;
                sh.hole[(it.seg + 8) & 15] = 0;
            }
            const bool go_on = it.seg == 0 || tc_wait(smem_u32(&sh.q_empty), (it.seg - 1) & 1, &sh.fail, a.polls);
            if (!__all_sync(0xffffffffu, go_on)) break;
            tc_copy_queries<S, 128>(a, sh, it.cur, p);
            tc_copies_arrive(smem_u32(&sh.q_full));
        }
        int tile;
        const bool values = it.what(tile);
        int64_t at = -1;
        const int t = tile * S::KT + mine;
        if (t < it.cur.len) {
            const int lb = kv.block.div(t);
            const int blk = kv.tables[static_cast<int64_t>(it.cur.b) * kv.max_blocks + first_block + lb];
            if (kv.valid(blk))
                at = kv.at(blk, it.cur.s / a.row_tiles, t - lb * kv.block_size());
            else
                sh.hole[it.seg & 15] = 1;
        }
        const int slot = use % S::kSlots;
        const bool go_on =
            use < S::kSlots || tc_wait(smem_u32(&sh.empty[slot]), (use / S::kSlots - 1) & 1, &sh.fail, a.polls);
        if (!__all_sync(0xffffffffu, go_on) || use == withhold) break;
        const uint32_t dst = smem_u32(sh.slot[slot]);
        const T* pool = static_cast<const T*>(values ? kv.v : kv.k);
#pragma unroll
        for (int i = 0; i < S::KT / kStep; ++i) {
            const int64_t from = __shfl_sync(0xffffffffu, at, i * kOwn + lane / kPieces);
            const bool take = from >= 0 && col;
            const int r = r0 + i * kStep;
            cp_async16(dst + (c >> 3) * S::kPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4), pool + (take ? from + c * 8 : 0),
                       take);
        }
        tc_copies_arrive(smem_u32(&sh.full[slot]));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// What the copies wrote is shown to the tensor cores' proxy by a thread of its
// own: the fence takes some 300 cycles, which would otherwise stand between
// the products.
template <typename S, typename A>
__device__ void tc_show_role(const A& a, TcShared<S>& sh, const AttnCursor& cur, int n) {
    TcUses<S> it(cur, n);
    for (int use = 0; use < 2 * n; ++use, it.next(a)) {
        if (it.u == 0) {
            if (!tc_wait(smem_u32(&sh.q_full), it.seg & 1, &sh.fail, a.polls)) return;
            fence_proxy_async_smem();
            mbar_arrive(smem_u32(&sh.q_shown));
        }
        if (!tc_wait(smem_u32(&sh.full[use % S::kSlots]), (use / S::kSlots) & 1, &sh.fail, a.polls)) return;
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&sh.shown[use % S::kSlots]));
    }
}

// ------------------------------------------------------------------ products
// One warp a stream.  A product's issue waits for the one before it, so that
// one warp's waits and commits would all be idle time of the tensor cores; and
// the two take turns, an output product and the next scores at a time, because
// streams that share the tensor cores fall into step and then form their
// weights at the same time, while these idle (16 trees of 32 rows over 8192
// positions: one warp for both 134 us, two 153, two in turns 129; since products
// are issued at the tensor cores' pace, 64 trees of 17 rows behind a shared
// prefix: one warp 203 us, two in turns 175).  Item i of
// a segment's part belongs to stream i & 1 and
// tile i >> 1 (WIDE) or i.  A stream's next scores follow its output product,
// whose weights lie where they go: products of one thread run in order.
template <typename S, typename A>
__device__ void tc_mma_role(const A& a, const TcMaps& maps, TcShared<S>& sh, const TcLayout& lay, AttnCursor cur, int n,
                            int x, int lane) {
    const uint32_t tm = sh.tmem;
    const uint32_t ts = tm + x * 128, to = tm + 256 + x * S::DP;
    constexpr uint32_t kScores = tc_idesc(S::KT, false), kOutputs = tc_idesc(S::DP, true);
    uint32_t p_seen = 0, turns = 0;
    int j0 = 0, seg = 0, use0 = 0, sent = -1;
    bool fine = true;  // no wait ran out; the same in all lanes
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        fine = __all_sync(0xffffffffu, fine && tc_wait(smem_u32(bar), parity, &sh.fail, a.polls));
    };
    // A slot is waited for in the order of use: its filling before (kSlots uses earlier) was then waited for too, so that
    // the parity tells the right one.  WIDE, a warp waits for every slot itself; else the other warp has waited for those
    // between, and this one has to be in its turn.
    auto wait_slot = [&](int use) {
        const int slot = use % S::kSlots;
        wait(S::TMA ? &sh.full[slot] : &sh.shown[slot], (use / S::kSlots) & 1);
        return slot;
    };
    while (fine && j0 < n) {
        const int nt = tc_part(cur, n - j0);
        const int items = nt * S::kTiles;
        const uint64_t qd = tc_desc_rows(smem_u32(sh.q) + (S::WIDE ? x * S::kSlot : 0), 1024);
        auto scores = [&](int slot) {
            const uint64_t kd = tc_desc_rows(smem_u32(sh.slot[slot]), lay.step);
#pragma unroll
            for (int kk = 0; kk < S::DP / 16; ++kk)
                tc_mma_ss(ts, qd + (((kk >> 2) * S::kPanel + (kk & 3) * 32) >> 4),
                          kd + (((kk >> 2) * lay.panel + (kk & 3) * 32) >> 4), kScores, kk > 0);
        };
        if (S::TMA && x == 0) {
            if (seg > 0) wait(&sh.q_empty, (seg - 1) & 1);
            if (!fine) break;
            tc_queries(a, maps, sh, cur, lane);
            sent = seg;
        }
        wait(&sh.q_shown, seg & 1);  // (both warps are through with the part before)
        if (x < items) {
            const int slot = wait_slot(use0 + S::keys_at(S::WIDE ? 0 : x, nt));
            if (!fine) break;
            tc_after_sync();
            if (tc_elect()) {
                scores(slot);
                tc_commit(smem_u32(&sh.s_full[x]));
                tc_commit(smem_u32(&sh.empty[slot]));
            }
            __syncwarp();
        }
        for (int i = x; i < items; i += 2) {
            const int t = S::WIDE ? i >> 1 : i;
            const bool more = i + 2 < items;
            int v_slot = 0, k_slot = 0;
            auto wait_slots = [&] {
                v_slot = wait_slot(use0 + S::values_at(t, nt));
                if (more) k_slot = wait_slot(use0 + S::keys_at(t + S::kLead, nt));
            };
            if (S::WIDE) wait_slots();
            if (i > 0) {
                wait(&sh.turn[x], turns & 1);
                ++turns;
            }
            if (!S::WIDE) wait_slots();
            // weights of the tile's first half, and then of the second
            const uint64_t vd = tc_desc_cols(smem_u32(sh.slot[v_slot]), lay.step, lay.panel);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                wait(half ? &sh.p_ready[x] : &sh.p_half[x], p_seen & 1);
                if (!fine) break;
                tc_after_sync();
                if (tc_elect()) {
#pragma unroll
                    for (int kk = half * S::KT / 32; kk < (half + 1) * S::KT / 32; ++kk)
                        tc_mma_ts(to, ts + kk * 8, vd + kk * (2 * lay.step >> 4), kOutputs, i >= 2 || kk > 0);
                    if (half) {
                        if (more) scores(k_slot);
                        if (i + 1 < items) mbar_arrive(smem_u32(&sh.turn[x ^ 1]));
                        tc_commit(smem_u32(more ? &sh.s_full[x] : &sh.o_done[x]));
                        tc_commit(smem_u32(&sh.empty[v_slot]));
                        if (more) tc_commit(smem_u32(&sh.empty[k_slot]));
                    }
                }
                __syncwarp();
            }
            if (!fine) break;
            ++p_seen;
        }
        if (tc_elect()) tc_commit(smem_u32(&sh.q_empty));
        __syncwarp();
        j0 += nt;
        use0 += 2 * nt;
        cur.tile += nt - 1;
        cur.next(a, S::KT);
        ++seg;
    }
    // nothing of this warp's is in flight when tensor memory is freed
    if (tc_elect()) tc_commit(smem_u32(&sh.end[x]));
    __syncwarp();
    mbar_wait_bounded(smem_u32(&sh.end[x]), 0, 1u << 30);
    if (sent >= 0) mbar_wait_bounded(smem_u32(&sh.q_shown), sent & 1, 1u << 30);  // nor a box of queries
}

// ------------------------------------------------------------------ softmax
template <typename S, typename A>
__device__ void tc_softmax_role(const A& a, TcShared<S>& sh, const TcLayout& lay, AttnCursor cur, const AttnRun& run,
                                int x, int row) {
    const int n = run.n;
    using T = typename S::Type;
    const KvView& kv = a.kv;
    constexpr bool kParts = std::is_same_v<A, PartArgs>;
    const int lane = row & 31, cta = blockIdx.x;
    const auto work = attn_work_of(a, gridDim.x, S::TM, S::DP);
    const int first_block = attn_first_block(a), own = attn_own(a);
    const int m_rows = a.rows * static_cast<int>(a.group.d);
    const uint32_t lanes = static_cast<uint32_t>(row & ~31) << 16;
    const uint32_t ts = sh.tmem + x * 128 + lanes;
    const float scale = attn_scale(a.scale);
    const float hidden = scale < 0.0f ? INFINITY : -INFINITY;
    uint32_t s_seen = 0, o_seen = 0;
    int j0 = 0, seg = 0, use0 = 0;
    auto parent_of = [&](int b) {
        return a.parents && lane > 0 && lane < a.rows ? a.parents[static_cast<int64_t>(b) * (a.rows - 1) + lane - 1]
                                                      : lane - 2;
    };
    int next_parent = parent_of(cur.b);
    while (j0 < n) {
        const int nt = tc_part(cur, n - j0);
        const int items = nt * S::kTiles;
        const int first_tile = cur.tile;
        const int h = cur.s / a.row_tiles, rt = cur.s - h * a.row_tiles;
        const int grow = rt * S::TM + (S::WIDE ? x * 128 : 0) + row;
        const bool warp_in = grow - lane < m_rows;  // the warp has rows
        const int r = a.group.div(grow), gq = grow - r * static_cast<int>(a.group.d);
        const int base = cur.len - own;
        // the next part's sequence is read while this one is worked on
        AttnCursor ahead = cur;
        ahead.tile += nt - 1;
        if (j0 + nt < n) ahead.next(a, S::KT);
        const int parent = next_parent;
        next_parent = parent_of(ahead.b);
        uint32_t line = 0;
        bool tree_ok = true;
        if (own && (first_tile + nt) * S::KT > base) {
            int depth;
            tree_ok = warp_tree_of(parent, a.rows, lane, line, depth);
        }
        const uint32_t anc = __shfl_sync(0xffffffffu, line, r < a.rows ? r : 0);
        float m_run = -INFINITY, l_run = 0.0f;
        for (int i = x; i < items; i += 2) {
            const int t = S::WIDE ? i >> 1 : i, t0 = (first_tile + t) * S::KT;
            const bool fine = tc_wait(smem_u32(&sh.s_full[x]), s_seen & 1, &sh.fail, a.polls);
            ++s_seen;
            if (!__all_sync(0xffffffffu, fine)) break;
            tc_after_sync();
            const bool edge = t0 + S::KT > base;
            auto half_ready = [&] {
                tc_wait_st();
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.p_half[x]));
            };
            if (warp_in) {
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc_ld32(ts + c * 32, s[c]);
                tc_wait_ld();
                // positions that not every row sees: of 32 columns
                auto hide = [&](int c) {
                    // bit e: position t0 + 32 c + e is before the pass's rows, or one that this row sees
                    const int gap = base - (t0 + c * 32);
                    const uint32_t open = gap >= 32 ? ~0u
                                          : gap >= 0 ? (anc << gap) | ((1u << gap) - 1)
                                          : gap > -32 ? anc >> -gap
                                                      : 0u;
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(open >> e & 1)) s[c][e] = __float_as_uint(hidden);
                };
                if (edge) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) hide(c);
                }
                // weights of columns 64 half .., in bf16 for the product (relative 2^-8 each, random in sign); their sum is
                // of the fp32 ones
                uint32_t w[32];
                const f2 sc = pack2(scale, scale);
                auto weigh = [&](int half) {
                    const float m_use = m_run == -INFINITY ? 0.0f : m_run;
                    const f2 nm = pack2(-m_use, -m_use);
                    f2 sum[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t* p = &s[2 * half + (e >> 4)][2 * (e & 15)];
                        float w0, w1;
                        unpack2(fma2(pack2(__uint_as_float(p[0]), __uint_as_float(p[1])), sc, nm), w0, w1);
                        w0 = ex2(w0);
                        w1 = ex2(w1);
                        sum[e & 1] = add2(sum[e & 1], pack2(w0, w1));
                        w[e] = kv_pack_bf16(w0, w1);
                    }
                    float l0, l1;
                    unpack2(add2(sum[0], sum[1]), l0, l1);
                    return l0 + l1;
                };
                float top[4] = {hidden, hidden, hidden, hidden};
                if (scale >= 0.0f) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
#pragma unroll
                        for (int c = 0; c < 4; ++c) top[c] = max3(top[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                    top[0] = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 2)
#pragma unroll
                        for (int c = 0; c < 4; ++c) top[c] = min3(top[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
                    top[0] = fminf(fminf(top[0], top[1]), fminf(top[2], top[3]));
                }
                top[0] *= scale;
                // the running maximum moves only when a score passes it by 8 (weights stay below 2^8); rows behind the
                // last, whose queries are whatever shared memory held, have no say in it
                if (__any_sync(0xffffffffu, grow < m_rows && top[0] > m_run + 8.0f)) {
                    const float m_new = fmaxf(m_run, top[0]);
                    const float keep = m_new == -INFINITY ? 1.0f : ex2(m_run - m_new);
                    m_run = m_new;
                    l_run *= keep;
                    if (i != x) {
                        const uint32_t to = sh.tmem + 256 + x * S::DP + lanes;
#pragma unroll 1
                        for (int c = 0; c < S::DP / 16; ++c) {
                            uint32_t o[16];
                            tc_ld16(to + c * 16, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                            tc_st16(to + c * 16, o);
                        }
                    }
                }
                const float l_half = weigh(0);
                tc_st32(ts, w);
                if (!edge) half_ready();
                l_run += l_half;
                l_run += weigh(1);
                tc_st32(ts + 32, w);
                tc_wait_st();
            }
            if (cur.len > 0 && edge) {
                // values of the pass's rows that are not finite are taken out of the product, where a weight of zero
                // would not hide them; they are added to the rows that see them at the segment's end
                const int slot = (use0 + S::values_at(t, nt)) % S::kSlots;
                // (the filling before was used up: scores of this tile follow it)
                tc_wait(smem_u32(&sh.full[slot]), (use0 + S::values_at(t, nt)) / S::kSlots & 1, &sh.fail, a.polls);
                // (boxes bring the rest of the last block too, whatever it holds: zeros in its place)
                const int lo_r = base > t0 ? base - t0 : 0, end_r = cur.len - t0 < S::KT ? cur.len - t0 : S::KT;
                int hi_r = end_r;
                if (S::TMA && end_r < S::KT) {
                    hi_r = (kv.block.div(cur.len - 1) + 1) * kv.block_size() - t0;
                    if (hi_r > S::KT) hi_r = S::KT;
                }
                for (int y = lo_r * (S::DP / 8) + row; y < hi_r * (S::DP / 8); y += 128) {
                    const int vr = y / (S::DP / 8), vc = y % (S::DP / 8);
                    KvVec<T>* vx = reinterpret_cast<KvVec<T>*>(sh.slot[slot] + lay.at(vr, vc));
                    if (vr >= end_r) {
                        *reinterpret_cast<uint4*>(vx) = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    KvVec<T> v = *vx;
                    bool wild = false;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (!finite(KvType<T>::load(v.x[e]))) {
                            v.x[e] = KvType<T>::store(0.0f);
                            wild = true;
                        }
                    if (wild) {
                        // (noted before it is gone: with WIDE the other stream looks at the same values)
                        atomicOr(&sh.wild[seg & 15], 1u << (t0 + vr - base));
                        __threadfence_block();
                        *vx = v;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            // (values that the products must not see are gone before the first of them)
            if (!warp_in || edge) half_ready();
            tc_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.p_ready[x]));
        }
        // the segment's part ends
        if (items > x) {
            tc_wait(smem_u32(&sh.o_done[x]), o_seen & 1, &sh.fail, a.polls);
            ++o_seen;
        }
        __syncwarp();
        tc_after_sync();
        float e0 = 1.0f, e1 = 0.0f;  // factors of the two streams' outputs
        if constexpr (!S::WIDE) {
            sh.ml[x][row] = make_float2(m_run, l_run);
            __syncwarp();
            asm volatile("bar.sync 2, 256;" ::: "memory");
            tc_after_sync();
            const float2 one = sh.ml[0][row], two = sh.ml[1][row];
            m_run = fmaxf(one.x, two.x);
            const float m_use = m_run == -INFINITY ? 0.0f : m_run;
            e0 = ex2(one.x - m_use);
            e1 = ex2(two.x - m_use);
            l_run = one.y * e0 + two.y * e1;
        }
        const bool ends = first_tile + nt == cur.tiles;
        const bool whole = first_tile == 0 && ends;
        const int64_t piece = kParts && whole ? 2ll * gridDim.x + attn_seg(a, cur) : 2ll * cta + (first_tile == 0 ? 1 : 0);
        int status = cur.len < 0 ? KV_LENGTH : cur.len == 0 ? 0 : tree_ok ? 0 : KV_PARENT;
        if (sh.hole[seg & 15]) status |= KV_BLOCK;
        if (tc_failed(&sh.fail)) status |= KV_TIMEOUT;
        const bool zero = cur.len <= 0 || status != 0;
        const uint32_t seen = anc & sh.wild[seg & 15];
        const int64_t head = (static_cast<int64_t>(cur.b) * a.rows + r) * a.q_heads + static_cast<int64_t>(h) * a.group.d + gq;
        const float inv = 1.0f / l_run;
        if (warp_in) {
            // one row tile: each stream writes half of the columns
            constexpr int kCols = S::WIDE ? S::DP : S::DP / 2;
            const uint32_t to = sh.tmem + 256 + lanes;
#pragma unroll 1
            for (int c = 0; c < kCols / 32; ++c) {
                const int d0 = (S::WIDE ? 0 : x * kCols) + c * 32;
                if (d0 >= kv.dim) break;
                __syncwarp();
                float o[32];
                uint32_t t[32];
                tc_ld32(to + (S::WIDE ? x * S::DP : 0) + d0, t);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(t[e]);
                if constexpr (!S::WIDE) {
                    if (items > 1) {
                        tc_ld32(to + S::DP + d0, t);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = o[e] * e0 + __uint_as_float(t[e]) * e1;
                    }
                }
                if (grow < m_rows) {
                    for (uint32_t left = seen; left; left &= left - 1) {
                        const int pos = base + __ffs(left) - 1, lb = kv.block.div(pos);
                        const int blk = kv.tables[static_cast<int64_t>(cur.b) * kv.max_blocks + first_block + lb];
                        if (!kv.valid(blk)) continue;
                        const T* v = static_cast<const T*>(kv.v) + kv.at(blk, h, pos - lb * kv.block_size()) + d0;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float y = d0 + e < kv.dim ? KvType<T>::load(v[e]) : 0.0f;
                            if (!finite(y)) o[e] += y;
                        }
                    }
                    if (!kParts && whole) {
                        T* out = static_cast<T*>(a.out) + head * kv.dim + d0;
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            if (d0 + e >= kv.dim) break;
                            float y[8];
#pragma unroll
                            for (int f = 0; f < 8; ++f) y[f] = zero ? 0.0f : o[e + f] * inv;
                            *reinterpret_cast<uint4*>(out + e) = make_uint4(kv_pack_bf16(y[0], y[1]), kv_pack_bf16(y[2], y[3]),
                                                                            kv_pack_bf16(y[4], y[5]), kv_pack_bf16(y[6], y[7]));
                        }
                    } else {
                        float4* acc = work.acc + (piece * (S::DP / 4) + d0 / 4) * S::TM +
                                      (S::WIDE ? x * 128 : 0) + row;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            acc[e * S::TM] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            if (grow < m_rows && (S::WIDE || x == 0)) {
                if (kParts || !whole)
                    work.ml[piece * S::TM + (S::WIDE ? x * 128 : 0) + row] = make_float2(m_run, l_run);
                else if (a.lse)
                    a.lse[head] = zero ? -INFINITY : m_run * 0.693147181f + logf(l_run);
            }
        }
        if (x == 0 && row == 0) {
            if constexpr (kParts) {
                work.status[piece] = status;
                if (first_tile == 0)
                    work.segs[attn_seg(a, cur)] =
                        PartNote{cta, run.owner(run.unit(j0 + cur.tiles - 1, seg)) * a.side + cta % a.side};
            } else {
                if (first_tile == 0 && cur.s == 0 && a.row_status) a.row_status[cur.b] = status;
                if (!whole) {
                    work.status[piece] = status;
                    if (first_tile == 0) {
                        work.notes[cta].b = cur.b;
                        work.notes[cta].s = cur.s;
                        work.notes[cta].last = run.owner(run.unit(j0 + cur.tiles - 1, seg));
                    }
                }
            }
        }
        if constexpr (!S::WIDE) {
            __syncwarp();
            tc_before_sync();
            asm volatile("bar.sync 2, 256;" ::: "memory");  // both streams' outputs are read
        }
        j0 += nt;
        use0 += 2 * nt;
        cur = ahead;
        ++seg;
    }
}

// ------------------------------------------------------------------ two parts at a time
// The tensor cores bound the prefix's part, the memory the other: they run
// side by side where the prefix has as many tiles as the sequences or more.
// The sequences' part comes first and takes half of the CTAs (which read nearly
// as fast as all: 64 trees of 17 rows over 500..1000 positions of their own take
// 48 us on 76 SMs, 53 on 152); the prefix's CTAs have the other SMs at once,
// and those of the sequences when these are through, which their shorter runs
// take into account.  A tile of a sequence counts as 7/4 of the prefix's on all
// SMs, a segment's end as two tiles, a start as five (64 trees of 17 rows, 500..1000
// of their own behind 8192 positions, at heads of 64: 145 us; 1 instead of 7/4 154,
// 11/4 164; 1000..2000 behind 16384 252, 250 and 284).
struct TcShare {
    int ctas;
    AttnLate late;
};

template <typename S>
__device__ __forceinline__ TcShare tc_share(const AttnArgs&, AttnCut&) {
    return TcShare{static_cast<int>(gridDim.x), {}};
}
template <typename S>
__device__ TcShare tc_share(const PartArgs& a, AttnCut& sh) {
    TcShare share{static_cast<int>(gridDim.x), {}};
    const int prefix = a.lens ? attn_prefix(a.kv, *a.prefix_len, a.prefix_cap) : 0;
    if (prefix <= 0) return share;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t tiles = 0;  // of the sequences, of a segment each
    for (int b = tid; b < a.sequences; b += S::kThreads) {
        const int len = min(a.lens[b], INT32_MAX - 512);
        tiles += attn_tiles(len > prefix ? len - prefix : 0, S::KT);
    }
    for (int off = 16; off > 0; off >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, off);
    if (lane == 0) sh.share[warp] = tiles;
    __syncthreads();
    tiles = 0;
    for (int w = 0; w < S::kThreads / 32; ++w) tiles += sh.share[w];
    const int64_t own = tiles * a.own_segs;
    const int64_t all = static_cast<int64_t>(attn_tiles(prefix, S::KT)) * a.prefix_segs;
    if (all < own) return share;
    const int half = gridDim.x / 2;
    if (!a.late) {
        share.ctas = half;
    } else {
        share.late.early = (static_cast<int>(gridDim.x) - half) / a.side;
        const int64_t time = 5 + (own + 2ll * a.sequences * a.own_segs) * 7 / (4 * half);
        share.late.less = S::WIDE ? (time + 1) / 2 : time;
    }
    return share;
}

// ------------------------------------------------------------------ the kernel
template <typename S, typename A>
__global__ void __launch_bounds__(S::kThreads, 1) tree_attention_tc_kernel(const A a, const __grid_constant__ TcMaps maps) {
    extern __shared__ __align__(1024) unsigned char tc_smem[];
    TcShared<S>& sh = *reinterpret_cast<TcShared<S>*>(tc_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if constexpr (S::TMA) {
        if (tid < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(tid ? &maps.v : &maps.k) : "memory");
    }
    AttnCursor cur;
    cur.b = 0;
    if (!attn_waits_late(a)) attn_wait();
    // row tiles side by side share the positions' cut
    const int side = attn_side(a), line = blockIdx.x / side, beside = blockIdx.x - line * side;
    const TcShare share = tc_share<S>(a, sh.cut);
    const AttnRun run = attn_cut<S::kThreads, S::kCost>(a, sh.cut, S::KT, a.kv.heads * (side > 1 ? 1 : a.row_tiles), line,
                                                        share.ctas / side, cur, share.late);
    if (side > 1) cur.s = cur.s * side + beside;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid's end
    if (tid == 0) {
        AttnNote* note = attn_work_of(a, gridDim.x, S::TM, S::DP).notes + blockIdx.x;
        note->b = -1;
        note->failed = 0;
        note->b0 = cur.b;
        sh.start = cur;
    }
    const int n = run.n;
    if (n == 0) {
        if (attn_waits_late(a)) attn_wait();
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < S::kSlots; ++i) {
            mbar_init(smem_u32(&sh.full[i]), S::TMA ? 1 : 128);
            mbar_init(smem_u32(&sh.shown[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), S::kTiles);  // the streams that use it
        }
        mbar_init(smem_u32(&sh.q_full), 128);
        mbar_init(smem_u32(&sh.q_shown), S::TMA && !maps.q_rows ? 32 : 1);
        mbar_init(smem_u32(&sh.q_empty), 2);
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&sh.s_full[x]), 1);
            mbar_init(smem_u32(&sh.p_half[x]), 4);
            mbar_init(smem_u32(&sh.p_ready[x]), 4);
            mbar_init(smem_u32(&sh.o_done[x]), 1);
            mbar_init(smem_u32(&sh.turn[x]), 1);
            mbar_init(smem_u32(&sh.end[x]), 1);
        }
        fence_mbar_init();
        sh.fail = (smem_u32(tc_smem) & 1023) != 0;  // the swizzle goes by address bits: no product from another alignment
    }
    if (tid < 16) {
        sh.wild[tid] = 0;
        sh.hole[tid] = 0;
    }
    __syncwarp();
    if (warp == 8) tc_alloc(smem_u32(&sh.tmem), 512);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const TcLayout lay = tc_layout<S>(maps);
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kMany));
        tc_softmax_role<S>(a, sh, lay, cur, run, warp >> 2, tid & 127);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kFew));
        if (warp < 10) {
            tc_mma_role<S>(a, maps, sh, lay, cur, n, warp - 8, lane);
        } else if constexpr (S::TMA) {
            if (warp < 10 + S::kBoxWarps) tc_box_role<S>(a, maps, sh, cur, n, warp - 10, lane);
        } else {
            if (warp >= 12)
                tc_copy_role<S>(a, sh, cur, n, tid - 384);
            else if (warp == 10 && lane == 0)
                tc_show_role<S>(a, sh, cur, n);
        }
    }
    __syncwarp();
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    if (warp == 8) tc_dealloc(sh.tmem, 512);
    // told when every role is done: a wait may run out after the threads that end a segment have looked at the flag
    if (tid == 0 && tc_failed(&sh.fail)) {
        AttnCursor at = sh.start;
        for (int left = n, nt; (nt = tc_part(at, left)) < left; left -= nt) {
            at.tile += nt - 1;
            at.next(a, S::KT);
        }
        AttnNote* note = attn_work_of(a, gridDim.x, S::TM, S::DP).notes + blockIdx.x;
        note->b1 = at.b;
        note->failed = 1;
    }
    if (attn_waits_late(a)) attn_wait();
}

}  // namespace specv
