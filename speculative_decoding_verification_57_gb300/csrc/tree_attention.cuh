// tree_attention.cuh -- attention of a pass's rows (a chain or a tree of
// drafted tokens) over the paged cache.
//
// Row r of sequence b sees the positions before the pass's rows and, of
// these, itself and its ancestors.  o = sum_j p_j v_j / sum_j p_j with
// p_j = 2^(c q.k_j - m), c = scale log2(e), m a running maximum.  Parts over
// different positions (m, l = sum p, a = sum p v) join by
// m = max m_i, l = sum l_i 2^(m_i - m), a = sum a_i 2^(m_i - m).
//
// Work.  The query heads of a kv head and the pass's rows are one matrix of
// rows * group rows, in row tiles of TM; its product with the keys is cut
// into tiles of positions.  A segment is (sequence, kv head, row tile); all
// segments' tiles form one line, which is cut into equal runs, one a CTA, so
// that ragged lengths load every SM alike and a single long sequence is
// spread over all of them.  The cut is computed from seq_lens on the device
// by every CTA alike: no plan, no host copy, and a captured graph follows the
// lengths.  A segment inside one CTA's run is written at once; one that is
// cut leaves partial results in the workspace, which tree_attention_join
// adds up in position order.
//
// A tile comes by 16-byte cp.async into swizzled shared memory, two tiles
// ahead of the products, the block numbers of a tile one tile before that.
// Warps own positions (KW of each tile) and rows: every key and value is
// read from shared memory by the warps of its positions only, and the
// softmax state of a warp is its own until its segment ends.
//
// bf16 with up to 16 rows a kv head, bf16 with head_dim above 128, and fp32;
// the rest is in tree_attention_tc.cuh.  fp32 values enter the tensor cores as
// two tf32 parts, three products each.
//
// Measured (GB300, graph replays over sets of inputs of more than twice the L2;
// bytes counted once, of 6691 GB/s measured): single rows, 32/8 heads of 128 in
// bf16, for 8 sequences over 500..1000 positions 16.1 us, 23%; for 64 over
// 1000..2000 79.4 us, 75%; heads of 256, 64 sequences: single rows over 1000..2000
// (16/4 heads) 98 us, 61%, trees of 17 rows over 2048..4096 574 us, 22%, three
// row tiles reading the cache each; fp32 chains of 5, 12 heads of 64, for 8
// sequences over 500..1000 24.0 us, 24%, for 64 104 us, 43%, and 40 rows of a kv
// head over 120,000 positions 152 us for a floor of 18.  The short ones are bound by the chain launch, length, block, tile
// (about 8 us) and by the join (4.5 us); fp32 by instructions (to split keys
// and values) with 12 warps an SM.
#pragma once
#include <type_traits>

#include "kv_cache.cuh"
#include "ptx.cuh"

namespace specv {

struct AttnArgs {
    KvView kv;
    const void* q;
    int64_t q_stride;
    const int32_t* parents;
    void* out;
    float* lse;
    int32_t* row_status;
    unsigned char* workspace;
    FastDiv group;   // query heads of a kv head
    FastDiv filled;  // rows of a row tile that hold any (the first tile has the most)
    int q_heads, rows, batch;
    int row_tiles;
    float scale;
    int withhold;    // test hook (tcgen05 kernel): this slot use of CTA 0's run is not copied (-1: none)
    uint32_t polls;  // most polls of a wait
};

// A part of an attention whose parts join later (prefix_attention.cuh): every
// segment leaves its outputs, undivided, in the workspace.
struct PartArgs : AttnArgs {
    const int32_t* prefix;  // positions before it, whole blocks, are left to another part; NULL: this is that part, of one
                            // sequence whose length is the prefix's and whose rows are all sequences', in their order
    int prefix_cap;         // the most positions that the prefix's table holds
    int own;                // rows of the pass among a sequence's positions: `rows`, or of the prefix none
    int side;               // row tiles of a kv head that as many CTAs side by side take over the same positions; 1: none
    bool late;              // the second of the two parts: waits at its end for what the kernels before wrote
    // both parts at the same time (tcgen05 kernels): what each has to know of the other; `lens` NULL: one behind the other
    const int32_t *lens, *prefix_len;  // of the sequences, and the prefix's
    int sequences, own_segs;            // sequences, and segments of a sequence
    int prefix_segs;                    // segments of 128 rows of the prefix
};

// Factor of the scores in base 2.  A scale of zero still has to tell hidden
// positions (an infinite score) from the others: the smallest number there is,
// so that the largest scores differ by less than 2^-20 of a weight.
__host__ __device__ __forceinline__ float attn_scale(float scale) {
    return scale == 0.0f ? 1.40129846e-45f : scale * 1.44269504f;
}

// ------------------------------------------------------------------ the cut
// Positions of sequence b that are attended to; -1 if it is refused by its length.
__device__ __forceinline__ int attn_len(const AttnArgs& a, int b) {
    const int len = a.kv.lens[b];
    return len == 0 || (len >= a.rows && a.kv.fits(len)) ? len : -1;
}

// The shared prefix's length; -1 if it is none of whole blocks that its table holds.
__device__ __forceinline__ int attn_prefix(const KvView& kv, int len, int cap) {
    return len >= 0 && len <= cap && len == static_cast<int>(kv.block.div(len)) * kv.block_size() ? len : -1;
}
// Of a part: the positions behind the prefix, or those of the prefix.
__device__ __forceinline__ int attn_len(const PartArgs& a, int b) {
    const int len = a.kv.lens[b];
    if (!a.prefix) return attn_prefix(a.kv, len, a.prefix_cap);
    if (len == 0) return 0;
    const int skip = attn_prefix(a.kv, *a.prefix, a.prefix_cap);
    return skip >= 0 && len >= a.rows && len - a.rows >= skip && a.kv.fits(len) ? len - skip : -1;
}
// The first entry of the tables that is looked at (of sequences that are not refused).
__device__ __forceinline__ int attn_first_block(const AttnArgs&) { return 0; }
__device__ __forceinline__ int attn_first_block(const PartArgs& a) {
    return a.prefix ? static_cast<int>(a.kv.block.div(max(*a.prefix, 0))) : 0;
}
// What the kernels before wrote is waited for at a kernel's start; by a part
// launched behind another at its end.  The part before lets it start when all of its CTAs
// are through with that wait, so that whatever was written before the call is
// there; and a kernel behind this one finds both parts' results, as this one
// ends after the part before.
__device__ __forceinline__ bool attn_waits_late(const AttnArgs&) { return false; }
__device__ __forceinline__ bool attn_waits_late(const PartArgs& a) { return a.late; }
__device__ __forceinline__ void attn_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Rows of the pass that are the last positions of a sequence.
__device__ __forceinline__ int attn_own(const AttnArgs& a) { return a.rows; }
__device__ __forceinline__ int attn_own(const PartArgs& a) { return a.own; }

// CTAs side by side, each with a row tile of its own of the same positions.
__device__ __forceinline__ int attn_side(const AttnArgs&) { return 1; }
__device__ __forceinline__ int attn_side(const PartArgs& a) { return a.side; }

// An idle or refused sequence counts as a tile, whose CTA writes its zeros.
__device__ __forceinline__ int attn_tiles(int len, int tile) { return len <= 0 ? 1 : (len + tile - 1) / tile; }

// a / b for a >= 0, b > 0; by the 32-bit division, an eighth of the other's time, wherever it will do.
__device__ __forceinline__ int64_t attn_div(int64_t a, int b) {
    return a >> 31 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// Run of CTA c of n over a line of `units`, floor(units c / n), and the CTA that has unit x.
__device__ __forceinline__ int64_t attn_run(int64_t units, int c, int n) {
    const int64_t each = attn_div(units, n);
    return each * c + attn_div((units - each * n) * c, n);
}
__device__ __forceinline__ int attn_owner(int64_t units, int64_t x, int n) {
    return static_cast<int>(((x + 1) * n - 1) / units);
}

// Where a run stands on the line of tiles.
struct AttnCursor {
    int b, s, tile;  // sequence, segment of it (kv head * row_tiles + row tile), tile
    int tiles, len;  // of the sequence

    template <typename A>
    __device__ __forceinline__ void next(const A& a, int tile_keys) {
        next(a, tile_keys, attn_side(a), a.kv.heads * a.row_tiles);
    }
    // ... on a line of `segs` segments a sequence, of which every `side`-th is on it
    template <typename A>
    __device__ __forceinline__ void next(const A& a, int tile_keys, int side, int segs) {
        if (++tile < tiles) return;
        tile = 0;
        if ((s += side) < segs) return;
        s = 0;
        if (++b < a.batch) {
            len = attn_len(a, b);
            tiles = attn_tiles(len, tile_keys);
        }
    }
};

// Shared memory of attn_cut.
struct AttnCut {
    int64_t sum[32], share[32];
    int64_t tiles[2];  // of the sequences before that at the run's start, and end
    int b[2];
};

// A CTA's run.  The line is of units: the tiles, and behind each segment's
// last, where runs are long, some that stand for what a segment costs besides
// its tiles (its queries, its end) and hold nothing.
struct AttnRun {
    int64_t units;  // of the line
    int64_t first;  // the unit of the run's first tile
    int used;       // CTAs that have runs
    int n;          // tiles of the run
    int extra;      // units behind a segment's last tile
    int early;      // CTAs of longer runs, which the first `early_units` units are cut into; the others have the rest
    int64_t early_units;

    // unit of a tile `tiles` tiles and `segments` segments on from the first
    __device__ __forceinline__ int64_t unit(int tiles, int segments) const {
        return first + tiles + static_cast<int64_t>(extra) * segments;
    }
    __device__ __forceinline__ int64_t bound(int c) const {
        return c <= early ? attn_run(early_units, c, early)
                          : early_units + attn_run(units - early_units, c - early, used - early);
    }
    __device__ __forceinline__ int owner(int64_t x) const {
        return x < early_units ? attn_owner(early_units, x, early)
                               : early + attn_owner(units - early_units, x - early_units, used - early);
    }
};

// CTAs from `early` on start late, by the time of `less` units; 0: none does.
struct AttnLate {
    int early = 0;
    int64_t less = 0;
};

// The run of CTA `cta` of `ctas` on a line of `segs` segments a sequence, and
// the cursor at its first tile, by the whole CTA (THREADS threads, a multiple of 32).  COST: a segment's extra
// units, in tiles, where a run has eight tiles or more.  Up to 32 sequences
// every warp finds out by itself; with more, each thread has some of them.
template <int THREADS, int COST, typename A>
__device__ AttnRun attn_cut(const A& a, AttnCut& sh, int tile_keys, int segs, int cta, int ctas, AttnCursor& cur,
                            AttnLate late = {}) {
    constexpr int kEnds = COST > 0 ? 2 : 1;  // of the run, looked for among the sequences
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool small = a.batch <= 32;
    // the total
    int64_t sum = 0, mine = 0, incl = 0;
    int my_len = 0;
    if (small) {
        if (lane < a.batch) {
            my_len = attn_len(a, lane);
            mine = attn_tiles(my_len, tile_keys);
        }
        incl = mine;
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        sum = __shfl_sync(0xffffffffu, incl, 31);
    } else {
        for (int b = tid; b < a.batch; b += THREADS) {
            mine = attn_tiles(attn_len(a, b), tile_keys);
            sum += mine;
        }
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) sh.sum[warp] = sum;
        __syncthreads();
        sum = 0;
        for (int w = 0; w < THREADS / 32; ++w) sum += sh.sum[w];
    }
    AttnRun run;
    run.extra = COST > 0 && sum * segs >= 8ll * ctas ? COST : 0;
    run.units = (sum + static_cast<int64_t>(run.extra) * a.batch) * segs;
    run.used = static_cast<int>(run.units < ctas ? run.units : ctas);
    run.first = 0;
    run.n = 0;
    run.early = run.used;
    run.early_units = run.units;
    if (late.less > 0 && run.units >= 8ll * ctas) {
        // runs of `more` units, and of `less` fewer
        const int rest = ctas - late.early;
        const int64_t more = (run.units + rest * late.less) / ctas;
        run.early = late.early;
        if (more > late.less)
            run.early_units = run.units - rest * (more - late.less);
        else
            run.used = late.early;
    }
    if (cta >= run.used) return run;
    const int64_t ends[2] = {run.bound(cta), run.bound(cta + 1)};
    // the sequences that hold the run's ends, and the tiles of those before them
    int at_b[kEnds], at_len[kEnds];
    int64_t at_before[kEnds];
    if (small) {
        const int64_t start = (incl - mine + static_cast<int64_t>(run.extra) * lane) * segs;
        const int64_t end = start + (mine + run.extra) * segs;
#pragma unroll
        for (int i = 0; i < kEnds; ++i) {
            const uint32_t hit = __ballot_sync(0xffffffffu, mine > 0 && start <= ends[i] && ends[i] < end);
            at_b[i] = hit ? __ffs(hit) - 1 : 0;  // (none: the line's end)
            at_len[i] = __shfl_sync(0xffffffffu, my_len, at_b[i]);
            at_before[i] = __shfl_sync(0xffffffffu, incl - mine, at_b[i]);
        }
    } else {
        int64_t before = 0;
        for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
            const int b = b0 + tid;
            // (one load a thread serves both passes for up to THREADS sequences)
            if (a.batch > THREADS) mine = b < a.batch ? attn_tiles(attn_len(a, b), tile_keys) : 0;
            if (b >= a.batch) mine = 0;
            incl = mine;
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            __syncthreads();
            if (lane == 31) sh.sum[warp] = incl;
            __syncthreads();
            int64_t ahead = before;
            for (int w = 0; w < warp; ++w) ahead += sh.sum[w];
            const int64_t start = (ahead + incl - mine + static_cast<int64_t>(run.extra) * b) * segs;
            const int64_t end = start + (mine + run.extra) * segs;
#pragma unroll
            for (int i = 0; i < kEnds; ++i)
                if (mine > 0 && start <= ends[i] && ends[i] < end) {
                    sh.b[i] = b;
                    sh.tiles[i] = ahead + incl - mine;
                }
            for (int w = warp; w < THREADS / 32; ++w) ahead += sh.sum[w];
            before = ahead;
            if ((before + static_cast<int64_t>(run.extra) * (b0 + THREADS)) * segs > ends[kEnds - 1]) break;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kEnds; ++i) {
            at_b[i] = ends[i] < run.units ? sh.b[i] : 0;
            at_len[i] = attn_len(a, at_b[i]);
            at_before[i] = sh.tiles[i];
        }
    }
    // tiles before each end; the cursor at the first
    int64_t tiles[kEnds];
#pragma unroll
    for (int i = 0; i < kEnds; ++i) {
        const int t = attn_tiles(at_len[i], tile_keys);
        const int64_t off = ends[i] - (at_before[i] + static_cast<int64_t>(run.extra) * at_b[i]) * segs;
        const int s = static_cast<int>(attn_div(ends[i] < run.units ? off : 0, t + run.extra));
        const int at = static_cast<int>(off - static_cast<int64_t>(s) * (t + run.extra));
        tiles[i] = ends[i] < run.units ? at_before[i] * segs + static_cast<int64_t>(s) * t + (at < t ? at : t) : sum * segs;
        if (i > 0) continue;
        run.first = ends[0];
        cur.b = at_b[0];
        cur.s = s;
        cur.len = at_len[0];
        cur.tiles = t;
        cur.tile = at < t ? at : t - 1;
        if (at >= t) {  // in the units behind a segment's last tile: on to the next segment
            run.first += t + run.extra - at;
            cur.next(a, tile_keys, 1, segs);
        }
    }
    run.n = static_cast<int>(kEnds == 2 ? tiles[kEnds - 1] - tiles[0] : ends[1] - ends[0]);
    return run;
}

// ------------------------------------------------------------------ workspace
// For every CTA a note on the segment that starts in its run and goes on
// past it, and two partial results: [0] of the segment its run starts in the
// middle of, [1] of the segment it starts and does not finish.
struct alignas(16) AttnNote {
    int b, s;    // b < 0: none
    int last;    // the CTA with the segment's last tile
    int failed;  // a wait of the CTA ran out: sequences b0 .. b1, all that its run touches, may be wrong
    int b0, b1;
};

struct AttnWork {
    AttnNote* notes;   // [ctas]
    int* status;       // [ctas * 2]
    float2* ml;        // [ctas * 2][TM]: maximum and sum of the weights
    float4* acc;       // [ctas * 2][DP / 4][TM]: four columns of a row, rows side by side
};

__host__ __device__ inline int64_t attn_work_bytes(int ctas, int tm, int dp) {
    return static_cast<int64_t>(ctas) * (sizeof(AttnNote) + 2 * sizeof(int) + 2 * tm * (sizeof(float2) + dp * 4ll));
}

__host__ __device__ inline AttnWork attn_work(unsigned char* p, int ctas, int tm, int dp) {
    // each part before the last is a multiple of 16 bytes (so are tm and dp)
    AttnWork w;
    w.notes = reinterpret_cast<AttnNote*>(p);
    w.ml = reinterpret_cast<float2*>(w.notes + ctas);
    w.acc = reinterpret_cast<float4*>(w.ml + static_cast<int64_t>(ctas) * 2 * tm);
    w.status = reinterpret_cast<int*>(w.acc + static_cast<int64_t>(ctas) * 2 * tm * (dp / 4));
    return w;
}

// ... and of a part: a note for every segment, and behind the partial results
// those of segments that one CTA has whole.
struct alignas(8) PartNote {
    int first, last;  // the CTAs with the segment's first and last tiles
};

struct PartWork {
    AttnNote* notes;  // [ctas]: whether a wait of the CTA ran out
    PartNote* segs;   // [segs]
    int* status;      // [ctas * 2 + segs]
    float2* ml;
    float4* acc;
};

__host__ __device__ inline int64_t part_pieces(int ctas, int64_t segs) { return 2ll * ctas + segs; }

__host__ __device__ inline int64_t part_work_bytes(int ctas, int64_t segs, int tm, int dp) {
    const int64_t pieces = part_pieces(ctas, segs);
    return (ctas * static_cast<int64_t>(sizeof(AttnNote)) + pieces * tm * (sizeof(float2) + dp * 4ll) +
            segs * static_cast<int64_t>(sizeof(PartNote)) + pieces * static_cast<int64_t>(sizeof(int)) + 255) / 256 * 256;
}

__host__ __device__ inline PartWork part_work(unsigned char* p, int ctas, int64_t segs, int tm, int dp) {
    const int64_t pieces = part_pieces(ctas, segs);
    PartWork w;
    w.notes = reinterpret_cast<AttnNote*>(p);
    w.ml = reinterpret_cast<float2*>(w.notes + ctas);
    w.acc = reinterpret_cast<float4*>(w.ml + pieces * tm);
    w.segs = reinterpret_cast<PartNote*>(w.acc + pieces * tm * (dp / 4));
    w.status = reinterpret_cast<int*>(w.segs + segs);
    return w;
}

// Where a CTA leaves the results of its segments, for either kind of call.
__device__ __forceinline__ AttnWork attn_work_of(const AttnArgs& a, int ctas, int tm, int dp) {
    return attn_work(a.workspace, ctas, tm, dp);
}
__device__ __forceinline__ PartWork attn_work_of(const PartArgs& a, int ctas, int tm, int dp) {
    return part_work(a.workspace, ctas, static_cast<int64_t>(a.batch) * a.kv.heads * a.row_tiles, tm, dp);
}
__device__ __forceinline__ int64_t attn_seg(const AttnArgs& a, const AttnCursor& cur) {
    return static_cast<int64_t>(cur.b) * a.kv.heads * a.row_tiles + cur.s;
}

// ------------------------------------------------------------------ matrix instructions
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x = hi + lo with both in tf32 (11 significant bits each): a product of two
// such pairs without lo * lo is off by 3 * 2^-22 of its size.  What hi leaves
// has 12 bits, so that lo cut off is off by no more than lo rounded.  An x that
// rounds to infinity has an infinite hi, and lo, a difference, is infinite or no
// number.  END: hi is the largest tf32 number then, so that a finite x has two
// finite parts (which add up to no more than x) and an infinite one an infinite
// lo; but the instruction costs: in every split, 40 rows of fp32 over 120,000
// positions take 179 us, for the values only 152.
template <bool END = false>
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    if (END)
        asm("cvt.rna.satfinite.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    else
        asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}

// 16 bytes global -> shared; zeros if !take (src is then not read)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
    const int n = take ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void attn_store4(float* p, float a, float b, float c, float d) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void attn_store4(__nv_bfloat16* p, float a, float b, float c, float d) {
    *reinterpret_cast<uint2*>(p) = make_uint2(kv_pack_bf16(a, b), kv_pack_bf16(c, d));
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// ------------------------------------------------------------------ shapes
// DP: head_dim rounded up to 64, 128 or 256 (the columns past head_dim are
// zeros in shared memory); RG row groups of 16 a warp, WR warps over rows, 4
// over positions: a row tile of TM = 16 RG WR rows.
template <typename T, int DP_, int RG_, int WR_>
struct AttnShape {
    using Type = T;
    static constexpr bool kBf16 = sizeof(T) == 2;
    static constexpr int DP = DP_, RG = RG_, WR = WR_, WK = 4;
    static constexpr int TM = 16 * RG * WR;
    static constexpr int KW = kBf16 ? 16 : 8;  // positions of a warp in a tile: the k of its matrix instruction
    static constexpr int KT = KW * WK;         // positions of a tile
    static constexpr int kThreads = 32 * WR * WK;
    static constexpr int kRow = DP * static_cast<int>(sizeof(T));  // bytes of a position
    static constexpr int kHalf = KT * kRow;                        // keys, or values, of a tile
    static constexpr int kStages = DP == 256 ? 2 : 3;
    static constexpr int kAhead = kStages - 1;
    static constexpr int kQ = TM * kRow;  // bytes of a row tile of queries
    static constexpr int kSmem = kStages * (2 * kHalf + kQ);
    // queries in registers for as long as a segment, unless the outputs need these
    static constexpr bool kQRegs = kBf16 && RG * DP <= 128;
    static constexpr bool kQSplit = !kBf16 && RG * DP <= 64;  // ... as their two tf32 parts
    // resident CTAs: by shared memory (227 KB, 1 KB a CTA taken, about 3 KB
    // static) and by registers (outputs, queries, and about 100 others)
    static constexpr int kFit = 227 * 1024 / (kSmem + 4096);
    static constexpr int kRegs = RG * DP / 2 + (kQRegs ? RG * DP / 4 : kQSplit ? RG * DP - 30 : 0) + 100;
    static constexpr int kMost = 65536 / (kRegs * kThreads) > 1 ? 65536 / (kRegs * kThreads) : 1;
    static constexpr int kCtas = kFit > kMost ? kMost : kFit;
    // a segment's end adds up the position warps' results in the tile last consumed, so many of them side by side
    static constexpr int kSide = 2 * kHalf / (TM * DP * 4) > 4 ? 4 : 2 * kHalf / (TM * DP * 4);
    static_assert(kSide == 1 || kSide == 2 || kSide == 4, "the reduction fits a stage");
};

// Byte offset of 16-byte piece c of row r: pieces change places within a row
// by the row, so that eight rows of the same piece lie in different banks.
template <typename S>
__device__ __forceinline__ uint32_t attn_at(int r, int c) {
    return static_cast<uint32_t>(r * S::kRow + ((c ^ (r & 7)) << 4));
}

// Product of query row m (at sq) and position n (at sk) of fp32 tiles, summed
// in float64, whose range no sum of such products leaves.
template <typename S>
__device__ float attn_dot(uint32_t sq, int m, uint32_t sk, int n) {
    double sum = 0.0;
#pragma unroll 1
    for (int c = 0; c < S::DP; ++c)
        sum += static_cast<double>(ld_shared_f32(sq + attn_at<S>(m, c >> 2) + (c & 3) * 4)) *
               static_cast<double>(ld_shared_f32(sk + attn_at<S>(n, c >> 2) + (c & 3) * 4));
    return static_cast<float>(sum);
}

// ------------------------------------------------------------------ the kernel
template <typename S, typename A>
__global__ void __launch_bounds__(S::kThreads, S::kCtas) tree_attention_kernel(const A a) {
    constexpr bool kParts = std::is_same_v<A, PartArgs>;
    using T = typename S::Type;
    constexpr int DP = S::DP, RG = S::RG, KT = S::KT, KW = S::KW, TM = S::TM, kStages = S::kStages, kAhead = S::kAhead;
    constexpr int kVec = KvType<T>::kVec;
    constexpr int kPieces = DP / kVec;  // 16-byte pieces of a position
    constexpr int NT = DP / 8;          // 8-wide column tiles of the output
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t s_row[2][KT];                 // where the positions of a tile lie (< 0: nowhere)
    __shared__ int s_hole[4][KT / 32 > 0 ? KT / 32 : 1];  // whether a position's block is outside the pool
    __shared__ int s_parents[kStages][32];
    __shared__ float2 s_ml[4][TM];
    __shared__ AttnCut s_cut;
    __shared__ uint32_t s_wild[2];  // nodes with values that are not finite, of a segment and the next
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wk = warp & 3, wr = warp >> 2;
    const int quad = lane >> 2, two = (lane & 3) * 2;
    const KvView& kv = a.kv;
    const int cta = blockIdx.x, ctas = gridDim.x;
    const auto work = attn_work_of(a, ctas, TM, DP);
    const uint32_t base_s = smem_u32(smem);
    const int m_rows = a.rows * static_cast<int>(a.group.d);  // rows of a kv head
    const float c_scale = attn_scale(a.scale);
    const float hidden = c_scale < 0.0f ? INFINITY : -INFINITY;

    AttnCursor cur, ahead, ids;
    if (!attn_waits_late(a)) attn_wait();
    const AttnRun run = attn_cut<S::kThreads, 0>(a, s_cut, KT, kv.heads * a.row_tiles, cta, ctas, cur);
    const int first_block = attn_first_block(a);
    if (tid == 0) {
        s_wild[0] = s_wild[1] = 0;
        work.notes[cta].b = -1;
        work.notes[cta].failed = 0;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join waits for this grid's end
    const int n = run.n;
    if (n == 0) {
        if (attn_waits_late(a)) attn_wait();
        return;
    }
    ids = ahead = cur;

    // block number of this thread's position in tile `i` of the run, whose cursor `ids` is: into a register ...
    struct Place {
        int blk, in, h;  // in: position in the block, < 0 for none
    };
    int ids_i = 0;
    auto fetch_row = [&]() {
        Place p = {0, -1, 0};
        if (ids_i < n) {
            const int t = ids.tile * KT + tid;
            if (tid < KT && t < ids.len) {
                const int lb = kv.block.div(t);
                // (no read-only load: the kernel may have started before the one that wrote the table ended)
                p.blk = kv.tables[static_cast<int64_t>(ids.b) * kv.max_blocks + first_block + lb];
                p.in = t - lb * kv.block_size();
                p.h = ids.s / a.row_tiles;
            }
            ids.next(a, KT);
        }
        ++ids_i;
        return p;
    };
    // ... and from there its place to shared memory, for the copies of tile i
    auto post_row = [&](int i, const Place& p) {
        if (tid < KT) {
            const bool valid = p.in >= 0 && kv.valid(p.blk);
            s_row[i & 1][tid] = valid ? kv.at(p.blk, p.h, p.in) : -1;
            const bool any = __any_sync(0xffffffffu, p.in >= 0 && !valid);
            if (lane == 0) s_hole[i & 3][warp] = any;
        }
    };
    // copies of tile i of the run (its cursor is `ahead`); the first tile of a segment brings its queries and parents
    int ahead_seg = 0;
    auto copy_tile = [&](int i) {
        if (i < n) {
            const uint32_t st = base_s + (i % kStages) * 2 * S::kHalf;
            const T* k = static_cast<const T*>(kv.k);
            const T* v = static_cast<const T*>(kv.v);
            const int row0 = tid / kPieces, c = tid % kPieces;
            constexpr int kStep = S::kThreads / kPieces;
#pragma unroll
            for (int r = row0; r < KT; r += kStep) {
                const int64_t at = s_row[i & 1][r];
                const bool take = at >= 0 && c * kVec < kv.dim;
                const int64_t off = take ? at + c * kVec : 0;
                const uint32_t dst = st + attn_at<S>(r, c);
                cp_async16(dst, k + off, take);
                cp_async16(dst + S::kHalf, v + off, take);
            }
            if (ahead.tile == 0 || i == 0) {
                const int slot = ahead_seg % kStages;
                const uint32_t sq = base_s + kStages * 2 * S::kHalf + slot * S::kQ;
                const int h = ahead.s / a.row_tiles, rt = ahead.s - h * a.row_tiles;
                const T* q = static_cast<const T*>(a.q);
                for (int m = row0; m < TM; m += kStep) {
                    const int row = rt * TM + m;
                    const bool take = row < m_rows && c * kVec < kv.dim;
                    const int r = a.group.div(row), g = row - r * static_cast<int>(a.group.d);
                    const int64_t off = (static_cast<int64_t>(ahead.b) * a.rows + r) * a.q_stride +
                                        (static_cast<int64_t>(h) * a.group.d + g) * kv.dim + c * kVec;
                    cp_async16(sq + attn_at<S>(m, c), q + (take ? off : 0), take);
                }
                if (a.parents && tid < a.rows - 1)
                    cp_async4(smem_u32(&s_parents[slot][tid]),
                              a.parents + static_cast<int64_t>(ahead.b) * (a.rows - 1) + tid);
                ++ahead_seg;
            }
            ahead.next(a, KT);
        }
        cp_commit();
    };

    // fill the pipeline
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

    float o[RG][NT][4];
    float m_run[RG][2], l_run[RG][2];
    uint32_t anc[RG][2];
    uint32_t qf[S::kQRegs ? RG : 1][S::kQRegs ? DP / 16 : 1][4];
    uint32_t qh[S::kQSplit ? RG : 1][S::kQSplit ? DP / 8 : 1][4], ql[S::kQSplit ? RG : 1][S::kQSplit ? DP / 8 : 1][4];
    int seg = 0, status = 0, first_tile = 0;

    for (int i = 0; i < n; ++i) {
        post_row(i + kAhead, place);
        place = fetch_row();
        cp_wait<kAhead - 1>();
        __syncthreads();
        copy_tile(i + kAhead);
        const uint32_t sk = base_s + (i % kStages) * 2 * S::kHalf, sv = sk + S::kHalf;
        const int slot = seg % kStages;
        const uint32_t sq = base_s + kStages * 2 * S::kHalf + slot * S::kQ;
        const int h = cur.s / a.row_tiles, rt = cur.s - h * a.row_tiles;
        if (cur.tile == 0 || i == 0) {  // a segment starts
            first_tile = cur.tile;
            if (tid == 0) s_wild[(seg + 1) & 1] = 0;
            status = cur.len < 0 ? KV_LENGTH : 0;
            uint32_t line;
            int depth;
            if (!warp_tree(a.parents ? s_parents[slot] : nullptr, a.rows, lane, line, depth) && cur.len > 0)
                status |= KV_PARENT;
#pragma unroll
            for (int g = 0; g < RG; ++g) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = rt * TM + (wr * RG + g) * 16 + quad + 8 * e;
                    anc[g][e] = __shfl_sync(0xffffffffu, line, a.group.div(row < m_rows ? row : 0));
                    m_run[g][e] = -INFINITY;
                    l_run[g][e] = 0.0f;
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[g][t][e] = 0.0f;
                if constexpr (S::kQSplit) {
#pragma unroll
                    for (int kk = 0; kk < DP / 8; ++kk)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            split_tf32(ld_shared_f32(sq + attn_at<S>((wr * RG + g) * 16 + quad + 8 * (e & 1),
                                                                     kk * 2 + (e >> 1)) +
                                                     (lane & 3) * 4),
                                       qh[g][kk][e], ql[g][kk][e]);
                }
                if constexpr (S::kQRegs) {
#pragma unroll
                    for (int kk = 0; kk < DP / 16; ++kk)
                        ldsm4(sq + attn_at<S>((wr * RG + g) * 16 + (lane & 15), kk * 2 + (lane >> 4)), qf[g][kk]);
                }
            }
        }
#pragma unroll
        for (int w = 0; w < (KT + 31) / 32; ++w)
            if (s_hole[i & 3][w]) status |= KV_BLOCK;
        const int t0 = cur.tile * KT, base = cur.len - attn_own(a);
        const bool edge = t0 + KT > base;  // positions that not every row sees
        if (edge && cur.len > 0) {
            // values of the pass's rows that are not finite are taken out of
            // the product, where a weight of zero would not hide them; they
            // are added to the rows that see them at the segment's end
            for (int x = tid; x < KT * kPieces; x += S::kThreads) {
                const int r = x / kPieces, t = t0 + r;
                if (t < base || t >= cur.len) continue;
                KvVec<T>* p = reinterpret_cast<KvVec<T>*>(smem + (sv - base_s) + attn_at<S>(r, x % kPieces));
                bool wild = false;
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (!finite(KvType<T>::load(p->x[e]))) {
                        p->x[e] = KvType<T>::store(0.0f);
                        wild = true;
                    }
                if (wild) atomicOr(&s_wild[seg & 1], 1u << (t - base));
            }
            __syncthreads();
        }
        // scores of this warp's positions
        constexpr int ST = KW / 8;
        float s[RG][ST][4];
#pragma unroll
        for (int g = 0; g < RG; ++g)
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[g][t][e] = 0.0f;
        if constexpr (S::kBf16) {
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                uint32_t kf[4];
                ldsm4(sk + attn_at<S>(wk * KW + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)), kf);
#pragma unroll
                for (int g = 0; g < RG; ++g) {
                    if constexpr (S::kQRegs) {
                        mma_bf16(s[g][0], qf[g][kk], kf[0], kf[1]);
                        mma_bf16(s[g][ST - 1], qf[g][kk], kf[2], kf[3]);
                    } else {
                        uint32_t qx[4];
                        ldsm4(sq + attn_at<S>((wr * RG + g) * 16 + (lane & 15), kk * 2 + (lane >> 4)), qx);
                        mma_bf16(s[g][0], qx, kf[0], kf[1]);
                        mma_bf16(s[g][ST - 1], qx, kf[2], kf[3]);
                    }
                }
            }
        } else {
            float s_low[RG][4] = {};
#pragma unroll(S::kQSplit ? DP / 8 : 4)
            for (int kk = 0; kk < DP / 8; ++kk) {
                uint32_t bh[2], bl[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    split_tf32(ld_shared_f32(sk + attn_at<S>(wk * KW + quad, kk * 2 + e) + (lane & 3) * 4), bh[e], bl[e]);
#pragma unroll
                for (int g = 0; g < RG; ++g) {
                    uint32_t ah[4], al[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (S::kQSplit) {
                            ah[e] = qh[g][kk][e];
                            al[e] = ql[g][kk][e];
                        } else {
                            split_tf32(ld_shared_f32(sq + attn_at<S>((wr * RG + g) * 16 + quad + 8 * (e & 1),
                                                                     kk * 2 + (e >> 1)) +
                                                     (lane & 3) * 4),
                                       ah[e], al[e]);
                        }
                    }
                    // (the small products add up by themselves: a sum of the tensor cores loses bits of its size a step)
                    mma_tf32(s_low[g], al, bh[0], bh[1]);
                    mma_tf32(s_low[g], ah, bl[0], bl[1]);
                    mma_tf32(s[g][0], ah, bh[0], bh[1]);
                }
            }
#pragma unroll
            for (int g = 0; g < RG; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[g][0][e] += s_low[g][e];
            // a score that is not finite: infinities and values near the ends of the type, whose parts are infinite or no
            // numbers though the score need not be
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                if (finite(fabsf(s[g][0][0]) + fabsf(s[g][0][1]) + fabsf(s[g][0][2]) + fabsf(s[g][0][3]))) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!finite(s[g][0][e]))
                        s[g][0][e] = attn_dot<S>(sq, (wr * RG + g) * 16 + quad + 8 * (e >> 1), sk, wk * KW + two + (e & 1));
            }
        }
        // weights: the running maximum moves only when a score passes it by
        // 8 (weights stay below 2^8), so that the sums are seldom rescaled
#pragma unroll
        for (int g = 0; g < RG; ++g) {
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (edge) {
                        const int pos = t0 + wk * KW + t * 8 + two + (e & 1);
                        if (pos >= base && !(pos < cur.len && (anc[g][e >> 1] >> (pos - base) & 1))) s[g][t][e] = hidden;
                    }
                    top[e >> 1] = fmaxf(top[e >> 1], s[g][t][e] * c_scale);
                }
            bool move = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                move |= top[e] > m_run[g][e] + 8.0f;
            }
            if (__any_sync(0xffffffffu, move)) {
                float keep[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float m_new = fmaxf(m_run[g][e], top[e]);
                    keep[e] = m_new == -INFINITY ? 1.0f : ex2(m_run[g][e] - m_new);
                    m_run[g][e] = m_new;
                    l_run[g][e] *= keep[e];
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[g][t][e] *= keep[e >> 1];
            }
            const float m_use[2] = {m_run[g][0] == -INFINITY ? 0.0f : m_run[g][0],
                                    m_run[g][1] == -INFINITY ? 0.0f : m_run[g][1]};
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[g][t][e] = ex2(fmaf(s[g][t][e], c_scale, -m_use[e >> 1]));
                    l_run[g][e >> 1] += s[g][t][e];
                }
        }
        // weights times values; bf16 weights are rounded to bf16 for the
        // product (relative 2^-8 each, random in sign; the sum l is not)
        if constexpr (S::kBf16) {
            uint32_t pf[RG][4];
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                pf[g][0] = kv_pack_bf16(s[g][0][0], s[g][0][1]);
                pf[g][1] = kv_pack_bf16(s[g][0][2], s[g][0][3]);
                pf[g][2] = kv_pack_bf16(s[g][ST - 1][0], s[g][ST - 1][1]);
                pf[g][3] = kv_pack_bf16(s[g][ST - 1][2], s[g][ST - 1][3]);
            }
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                uint32_t vf[4];
                ldsm4t(sv + attn_at<S>(wk * KW + (lane & 15), t + (lane >> 4)), vf);
#pragma unroll
                for (int g = 0; g < RG; ++g) {
                    mma_bf16(o[g][t], pf[g], vf[0], vf[1]);
                    mma_bf16(o[g][t + 1], pf[g], vf[2], vf[3]);
                }
            }
        } else {
            uint32_t ph[RG][4], pl[RG][4];  // k of the instruction: position 2 (lane & 3), then the odd ones
#pragma unroll
            for (int g = 0; g < RG; ++g) {
                split_tf32(s[g][0][0], ph[g][0], pl[g][0]);
                split_tf32(s[g][0][2], ph[g][1], pl[g][1]);
                split_tf32(s[g][0][1], ph[g][2], pl[g][2]);
                split_tf32(s[g][0][3], ph[g][3], pl[g][3]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t bh[2], bl[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    split_tf32<true>(ld_shared_f32(sv + attn_at<S>(wk * KW + two + e, t * 2 + (quad >> 2)) + (quad & 3) * 4),
                                     bh[e], bl[e]);
#pragma unroll
                for (int g = 0; g < RG; ++g) {
                    float part[4] = {};  // the tile's, added in fp32 proper
                    mma_tf32(part, pl[g], bh[0], bh[1]);
                    mma_tf32(part, ph[g], bl[0], bl[1]);
                    mma_tf32(part, ph[g], bh[0], bh[1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[g][t][e] += part[e];
                }
            }
        }
        const bool ends = cur.tile + 1 == cur.tiles;
        if (ends || i + 1 == n) {
            // the segment's part ends: the four position warps' results join
            // in the tile just consumed
#pragma unroll
            for (int g = 0; g < RG; ++g)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l_run[g][e] += __shfl_xor_sync(0xffffffffu, l_run[g][e], 1);
                    l_run[g][e] += __shfl_xor_sync(0xffffffffu, l_run[g][e], 2);
                    if ((lane & 3) == 0)
                        s_ml[wk][(wr * RG + g) * 16 + quad + 8 * e] = make_float2(m_run[g][e], l_run[g][e]);
                }
            __syncthreads();
            float* red = reinterpret_cast<float*>(smem + (sk - base_s));
            float keep[RG][2];
#pragma unroll
            for (int g = 0; g < RG; ++g)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = (wr * RG + g) * 16 + quad + 8 * e;
                    float m = -INFINITY;
                    for (int w = 0; w < 4; ++w) m = fmaxf(m, s_ml[w][row].x);
                    keep[g][e] = m == -INFINITY ? 1.0f : ex2(m_run[g][e] - m);
                }
            float* mine = red + (wk % S::kSide) * TM * DP;
#pragma unroll
            for (int w = 0; w < 4 / S::kSide; ++w) {
                if (wk / S::kSide == w) {
#pragma unroll
                    for (int g = 0; g < RG; ++g)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float2* p = reinterpret_cast<float2*>(
                                    mine + ((wr * RG + g) * 16 + quad + 8 * e) * DP + ((t * 8 + two) ^ ((quad & 3) * 8)));
                                float2 x = w == 0 ? make_float2(0.0f, 0.0f) : *p;
                                x.x += o[g][t][2 * e] * keep[g][e];
                                x.y += o[g][t][2 * e + 1] * keep[g][e];
                                *p = x;
                            }
                }
                __syncthreads();
            }
            const bool whole = first_tile == 0 && ends;
            const int64_t piece = kParts && whole ? 2ll * ctas + attn_seg(a, cur) : 2ll * cta + (first_tile == 0 ? 1 : 0);
            const uint32_t wild = s_wild[seg & 1];
            constexpr int kGroup = S::kThreads / TM;  // threads of a row
            const int row = tid / kGroup, lane_r = tid % kGroup;
            float m = -INFINITY, l = 0.0f;
            for (int w = 0; w < 4; ++w) m = fmaxf(m, s_ml[w][row].x);
            for (int w = 0; w < 4; ++w) l += s_ml[w][row].y * (m == -INFINITY ? 1.0f : ex2(s_ml[w][row].x - m));
            const int grow = rt * TM + row;
            const int r = a.group.div(grow), gq = grow - r * static_cast<int>(a.group.d);
            const int64_t token = static_cast<int64_t>(cur.b) * a.rows + r;
            const int64_t head = token * a.q_heads + static_cast<int64_t>(h) * a.group.d + gq;
            const uint32_t seen = wild ? [&] {
                uint32_t line;
                int depth;
                warp_tree(a.parents ? s_parents[slot] : nullptr, a.rows, lane, line, depth);
                uint32_t mine = 0;
                for (int x = 0; x < 32; ++x) {
                    const uint32_t y = __shfl_sync(0xffffffffu, line, x);
                    if (x == r) mine = y;
                }
                return mine & wild;
            }()
                                       : 0;
            const bool zero = cur.len <= 0 || status != 0;
            if (grow < m_rows) {
                const float inv = 1.0f / l;
                for (int d = lane_r * 4; d < kv.dim; d += kGroup * 4) {
                    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < S::kSide; ++w) {
                        const float4 x4 =
                            *reinterpret_cast<const float4*>(red + (w * TM + row) * DP + (d ^ ((row & 3) * 8)));
                        x[0] += x4.x;
                        x[1] += x4.y;
                        x[2] += x4.z;
                        x[3] += x4.w;
                    }
                    if (seen) {
                        for (int j = 0; j < a.rows; ++j) {
                            if (!(seen >> j & 1)) continue;
                            const int t = base + j, lb = kv.block.div(t);
                            const int blk = kv.tables[static_cast<int64_t>(cur.b) * kv.max_blocks + first_block + lb];
                            if (!kv.valid(blk)) continue;
                            const T* v = static_cast<const T*>(kv.v) + kv.at(blk, h, t - lb * kv.block_size()) + d;
                            for (int e = 0; e < 4; ++e) {
                                const float y = KvType<T>::load(v[e]);
                                if (!finite(y)) x[e] += y;
                            }
                        }
                    }
                    if (!kParts && whole) {
                        T* out = static_cast<T*>(a.out) + head * kv.dim + d;
                        attn_store4(out, zero ? 0.0f : x[0] * inv, zero ? 0.0f : x[1] * inv, zero ? 0.0f : x[2] * inv,
                                    zero ? 0.0f : x[3] * inv);
                    } else {
                        work.acc[(piece * (DP / 4) + d / 4) * TM + row] =
                            make_float4(x[0], x[1], x[2], x[3]);
                    }
                }
                if (lane_r == 0) {
                    if (!kParts && whole) {
                        if (a.lse) a.lse[head] = zero ? -INFINITY : m * 0.693147181f + logf(l);
                    } else {
                        work.ml[piece * TM + row] = make_float2(m, l);
                    }
                }
            }
            if (tid == 0) {
                if constexpr (kParts) {
                    work.status[piece] = status;
                    if (first_tile == 0)
                        work.segs[attn_seg(a, cur)] =
                            PartNote{cta, run.owner(run.unit(i + cur.tiles - cur.tile - 1, seg))};
                } else {
                    if (first_tile == 0 && cur.s == 0 && a.row_status) a.row_status[cur.b] = status;
                    if (!whole) {
                        work.status[piece] = status;
                        if (first_tile == 0) {
                            work.notes[cta].b = cur.b;
                            work.notes[cta].s = cur.s;
                            work.notes[cta].last =
                                run.owner(run.unit(i + cur.tiles - cur.tile - 1, seg));
                        }
                    }
                }
            }
            ++seg;
        }
        cur.next(a, KT);
    }
    if (attn_waits_late(a)) attn_wait();
}

// ------------------------------------------------------------------ the join
constexpr int kJoinThreads = 128;

// COLS times four columns of a row a thread, rows side by side, of the segment
// that CTA blockIdx.x of the kernel before noted; PIECES pieces of it at a
// time.  Bound by latency, so that a thread has several loads in flight: of
// many columns where there are many segments, each cut in two or three, of
// many pieces where there are few, each spread over many CTAs.
template <typename S, int PIECES, int COLS>
__global__ void __launch_bounds__(kJoinThreads) tree_attention_join(const AttnArgs a, int ctas) {
    using T = typename S::Type;
    constexpr int TM = S::TM, DP = S::DP;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const AttnWork work = attn_work(a.workspace, ctas, TM, DP);
    const int cta = blockIdx.x;
    const AttnNote note = work.notes[cta];
    if (note.failed && blockIdx.y == 0 && a.row_status)
        for (int b = note.b0 + static_cast<int>(threadIdx.x); b <= note.b1; b += kJoinThreads)
            atomicOr(a.row_status + b, KV_TIMEOUT);
    if (note.b < 0) return;
    const KvView& kv = a.kv;
    const int at = blockIdx.y * kJoinThreads + threadIdx.x;
    const int part = a.filled.div(at), row = at - part * static_cast<int>(a.filled.d);
    const int col = part * COLS;  // the first group of four columns
    const int h = note.s / a.row_tiles, rt = note.s - h * a.row_tiles;
    const int grow = rt * TM + row;
    if (col * 4 >= kv.dim || grow >= a.rows * static_cast<int>(a.group.d)) return;
    int status = 0;
    float m = -INFINITY, l = 0.0f;
    float4 x[COLS];
#pragma unroll
    for (int k = 0; k < COLS; ++k) x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c = cta; c <= note.last; c += PIECES) {
        float2 ml[PIECES];
        float4 y[PIECES][COLS];
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            ml[u] = make_float2(-INFINITY, 0.0f);
            if (c + u <= note.last) {
                // [1] of the CTA that starts the segment, then [0] of the next ones
                const int64_t piece = 2ll * (c + u) + (c + u == cta);
                status |= work.status[piece];
                ml[u] = work.ml[piece * TM + row];
#pragma unroll
                for (int k = 0; k < COLS; ++k) y[u][k] = work.acc[(piece * (DP / 4) + col + k) * TM + row];
            }
        }
        float m_new = m;
#pragma unroll
        for (int u = 0; u < PIECES; ++u) m_new = fmaxf(m_new, ml[u].x);
        const float m_use = m_new == -INFINITY ? 0.0f : m_new;
        const float before = ex2(m - m_use);
        m = m_new;
        l *= before;
#pragma unroll
        for (int k = 0; k < COLS; ++k)
            x[k] = make_float4(x[k].x * before, x[k].y * before, x[k].z * before, x[k].w * before);
#pragma unroll
        for (int u = 0; u < PIECES; ++u) {
            if (c + u > note.last) break;
            const float w = ex2(ml[u].x - m_use);
            l = fmaf(ml[u].y, w, l);
#pragma unroll
            for (int k = 0; k < COLS; ++k)
                x[k] = make_float4(fmaf(y[u][k].x, w, x[k].x), fmaf(y[u][k].y, w, x[k].y), fmaf(y[u][k].z, w, x[k].z),
                                   fmaf(y[u][k].w, w, x[k].w));
        }
    }
    if (at == 0 && note.s == 0 && status && a.row_status) atomicOr(a.row_status + note.b, status);
    const int r = a.group.div(grow), g = grow - r * static_cast<int>(a.group.d);
    const int64_t token = static_cast<int64_t>(note.b) * a.rows + r;
    const int64_t head = token * a.q_heads + static_cast<int64_t>(h) * a.group.d + g;
    const float inv = status ? 0.0f : 1.0f / l;
#pragma unroll
    for (int k = 0; k < COLS; ++k) {
        if (status) x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        attn_store4(static_cast<T*>(a.out) + head * kv.dim + (col + k) * 4, x[k].x * inv, x[k].y * inv, x[k].z * inv,
                    x[k].w * inv);
    }
    if (col == 0 && a.lse) a.lse[head] = status ? -INFINITY : m * 0.693147181f + logf(l);
}

}  // namespace specv
