// cache_evict.cuh -- sequences of a paged cache brought back to a budget of
// positions: per layer and kv head the first `first` and the last `recent`
// positions stay, and of those between the ones that gathered the largest
// mass (attention_mass.cuh), equal ones by the lowest position.
//
// With `line` = budget - recent, kept positions below the line stay where
// they are; the i-th hole below it takes the i-th kept position above it; the
// recent ones follow from the line on in their order.  Attention does not ask
// for an order of the positions before a pass (their rotation is in the
// keys), so that no more moves than that: a stable order would move nearly
// every kept position of a head.
//
// A CTA, or where there are few heads some side by side, has a row of masses
// (a layer, sequence and kv head).  CTAs of one row find the kept set each by
// itself and move columns of their own of the keys or the values, so that they
// need not meet; masses and lengths go to other memory than they come from.
// The least kept mass is found by its bits, eight at a time, from the top, and
// no further than it takes to tell the kept ones; moves are listed in position
// order by ballots and a scan over the warps' counts.  A thread has the masses
// of eight positions in registers.  Moves run in order, 16 bytes a thread and
// row, all loads of a step before its stores: a step's stores go to places that
// no later step reads, as sources of kept positions lie above the line and the
// recent ones, behind them, move down.
//
// A list has 1024 moves; the next one is found where it ended.  Every list used to be
// found among all positions, so that 131072 of them took 7.0 ms to 32768 (8 heads of
// 128 of 8 sequences, one layer) and take 1.9, most of it the first look, of 64 spans,
// at each row.  Masses of up to 2048 positions are read once for the choice, longer
// rows' once for each digit and list, and both again where they are moved.
//
// Measured (GB300, graph replays over sets of inputs beyond the L2; 8 heads of 128
// in bf16, budget 1024, 256 recent, up to twice as long before): 8 layers of 32
// sequences 158 us, 92% of 6803 GB/s; one layer of 8 sequences 14.7 us, a chain
// of length and blocks (2.8 us), the least mass (2.8), lists (2.9) and moves (6).
// Four pieces a thread in flight (two: 176 us, eight: 221, which spills), four CTAs
// an SM (five or six: 201 and 195), eight masses a thread (16, which spill: 212).
#pragma once
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace specv {

constexpr int kEvictThreads = 256;
constexpr int kEvictMoves = 1024;  // listed at a time
constexpr int kEvictAhead = 4;     // of a thread, in flight
constexpr int kEvictItems = 8;    // masses of a thread, kEvictThreads positions apart
constexpr int kEvictSpan = kEvictThreads * kEvictItems;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictMost = INT32_MAX - 4095;  // positions of a sequence: a span behind them is still an int

struct EvictArgs {
    KvView kv;
    const float* mass;  // [layers, B, heads, width]
    float* mass_out;
    int32_t* lens_out;
    int32_t* evicted;
    int32_t* row_status;
    int64_t layer_stride, width;
    int batch;
    int budget, recent, first;
    int split;          // CTAs of a row: 1, or some for the columns of the keys and as many for those of the values
    int pieces;         // of 16 bytes a CTA moves of a row
    FastDiv piece_div;  // by pieces
    int vec_elems;
};

// Masses as whole numbers in the same order; zeros alike, what is no number above all others.
__device__ __forceinline__ uint32_t evict_key(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

static_assert(kEvictSpan <= 4095 && kEvictMoves <= 4095 && 8 * kEvictThreads <= 4095, "counters of positions stay ints");

// The positions from `base` on: how many equal to the key, holes and kept ones above the line lie before.
struct EvictCount {
    int base;
    uint32_t equal, holes, above;
};

struct EvictShared {
    uint32_t hist[kEvictWarps][256];
    uint32_t count[kEvictItems * kEvictWarps];  // of a span, by item and warp: in position order
    uint32_t warp_sum[kEvictWarps];
    uint32_t total;
    uint32_t key, more, equal;  // the digits found so far, how many of those equal to them are kept, and how many there are
    EvictCount hole_at, above_at;  // where the lists of the next moves start
    int src[kEvictMoves], dst[kEvictMoves];
    int64_t from[kEvictMoves], to[kEvictMoves];
};

// Keys of the positions base + tid, base + tid + kEvictThreads, ..: those of n.
__device__ __forceinline__ void evict_load(const float* mass, int n, int base, uint32_t (&k)[kEvictItems]) {
#pragma unroll
    for (int j = 0; j < kEvictItems; ++j) {
        const int i = base + j * kEvictThreads + static_cast<int>(threadIdx.x);
        k[j] = 0;
        if (i < n) k[j] = evict_key(mass[i]);
    }
}

// sh.count (a barrier before) as exclusive sums, and their total; packed counts below 2^16 too.
__device__ __forceinline__ void evict_scan(EvictShared& sh) {
    static_assert(kEvictItems * kEvictWarps <= kEvictThreads, "a count a thread");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t v = tid < kEvictItems * kEvictWarps ? sh.count[tid] : 0;
    uint32_t incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += sh.warp_sum[w];
    if (tid < kEvictItems * kEvictWarps) sh.count[tid] = incl - v;
    if (tid == kEvictThreads - 1) sh.total = incl;
    __syncthreads();
}

// The `many`-th largest of n masses (1 <= many < n), as far as it takes:
// kept are keys above sh.key, and sh.more of the sh.equal ones equal to it.
// k: the first span's keys.
__device__ inline void evict_select(EvictShared& sh, const float* mass, int n, uint32_t many, uint32_t (&k)[kEvictItems]) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t key = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = lane; i < 256; i += 32) sh.hist[warp][i] = 0;
        __syncwarp();
        const uint32_t above = shift == 24 ? 0u : ~0u << (shift + 8);
        for (int base = 0; base < n; base += kEvictSpan) {
            if (n > kEvictSpan) evict_load(mass, n, base, k);
#pragma unroll
            for (int j = 0; j < kEvictItems; ++j) {
                if (base + j * kEvictThreads >= n) break;
                if (base + j * kEvictThreads + tid < n && (k[j] & above) == key)
                    atomicAdd(&sh.hist[warp][k[j] >> shift & 255], 1u);
            }
        }
        __syncthreads();
        // the digit in which the counts from the top pass `many`: thread t has digit 255 - t
        uint32_t c = 0;
#pragma unroll
        for (int w = 0; w < kEvictWarps; ++w) c += sh.hist[w][255 - tid];
        uint32_t incl = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += o;
        }
        if (lane == 31) sh.warp_sum[warp] = incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += sh.warp_sum[w];
        if (incl >= many && incl - c < many) {
            sh.key = key | static_cast<uint32_t>(255 - tid) << shift;
            sh.more = many - (incl - c);
            sh.equal = c;
        }
        __syncthreads();
        key = sh.key;
        many = sh.more;
        if (many == sh.equal) {  // all with these digits are kept: those above the key before them
            __syncthreads();
            if (tid == 0) {
                sh.key = key - 1;  // (not of 0, above which all are kept: `many` is below n)
                sh.more = 0;
            }
            __syncthreads();
            return;
        }
    }
}

__global__ void __launch_bounds__(kEvictThreads, 4) cache_evict_kernel(const EvictArgs e) {
    __shared__ EvictShared sh;
    const int tid = threadIdx.x;
    const KvView& kv = e.kv;
    const int part = blockIdx.x % e.split;
    const int64_t row = blockIdx.x / e.split;  // (layer * batch + b) * heads + h
    const int h = static_cast<int>(row % kv.heads), b = static_cast<int>(row / kv.heads % e.batch);
    const int layer = static_cast<int>(row / kv.heads / e.batch);
    const int len = kv.lens[b];
    int status = len < 0 || !kv.fits(len) || len > kEvictMost || len > e.width ? KV_LENGTH : 0;
    const bool over = status == 0 && len > e.budget;
    const int32_t* table = kv.tables + static_cast<int64_t>(b) * kv.max_blocks;
    if (over) {
        bool hole = false;
        for (int i = kv.block.div(e.first) + tid, last = kv.block.div(len - 1); i <= last; i += kEvictThreads)
            hole |= !kv.valid(table[i]);
        if (__syncthreads_or(hole)) status |= KV_BLOCK;
    }
    if (tid == 0 && part == 0 && layer == 0 && h == 0) {
        const bool cut = over && status == 0;
        e.lens_out[b] = cut ? e.budget : len;
        if (e.evicted) e.evicted[b] = cut ? len - e.budget : 0;
        if (e.row_status) e.row_status[b] = status;
    }
    const float* mass = e.mass + row * e.width;
    float* mass_out = e.mass_out + row * e.width;
    if (status != 0 || !over) {
        if (status == 0)
            for (int i = tid + part * kEvictThreads; i < len; i += kEvictThreads * e.split) mass_out[i] = mass[i];
        return;
    }
    const int line = e.budget - e.recent, many = line - e.first, tail = len - e.recent;
    const int n = tail - e.first;  // positions to choose from: more than `many`
    if (part == 0)  // (what lies in holes is written over below, behind barriers)
        for (int i = tid; i < line; i += kEvictThreads) mass_out[i] = mass[i];
    uint32_t key = 0, ties = 0, k[kEvictItems];  // kept: above key, or one of the first `ties` equal to it
    if (many > 0) {
        evict_load(mass + e.first, n, 0, k);
        evict_select(sh, mass + e.first, n, static_cast<uint32_t>(many), k);
        key = sh.key;
        ties = sh.more;
    }
    // the moves of rank [round, round + kEvictMoves): first those that fill holes, then the recent ones
    const int lane = tid & 31, warp = tid >> 5;
    const int parts = e.split > 1 ? 1 : 2;  // one CTA moves keys and then values
    unsigned char* pool = static_cast<unsigned char*>(e.split > 1 && (part & 1) ? kv.v : kv.k);
    const int64_t elem = 16 / e.vec_elems;
    const int64_t head_at = layer * e.layer_stride + static_cast<int64_t>(h) * kv.block_size() * kv.dim;
    const int64_t column = static_cast<int64_t>(part >> 1) * e.pieces * 16;
    int fills = many > 0 ? INT32_MAX : 0;
    for (int round = 0;; round += kEvictMoves) {
        // holes below the line and kept positions above it, by their ranks; both lists are as long.  The first time all
        // positions are looked at; then the holes from where the last list of them ended, and the others from there
        const int stop = round + kEvictMoves;
        for (int above_line = 0; round < fills && above_line < (round ? 2 : 1); ++above_line) {
            EvictCount at = {};
            if (round) at = above_line ? sh.above_at : sh.hole_at;
            const int end = round && !above_line ? many : n;
            while (at.base < end && (round == 0 || (above_line ? at.above : at.holes) < static_cast<uint32_t>(stop))) {
                const int base = at.base;
                if (tid == 0 && n > kEvictSpan) {  // (read behind the barriers below; a span has one list's moves at most)
                    if (at.holes <= static_cast<uint32_t>(stop) && !above_line) sh.hole_at = at;
                    if (at.above <= static_cast<uint32_t>(stop) && (above_line || round == 0)) sh.above_at = at;
                }
                if (n > kEvictSpan) evict_load(mass + e.first, n, base, k);
                uint32_t kept = 0, move = 0;  // of the thread's items
                if (ties > 0) {  // equal ones by their order
#pragma unroll
                    for (int j = 0; j < kEvictItems; ++j) {
                        if (lane == 0) sh.count[j * kEvictWarps + warp] = 0;
                        if (base + j * kEvictThreads >= n) continue;
                        const bool same = base + j * kEvictThreads + tid < n && k[j] == key;
                        const uint32_t all = __ballot_sync(0xffffffffu, same);
                        if (lane == 0) sh.count[j * kEvictWarps + warp] = __popc(all);
                        if (same) kept |= 1u << j;
                    }
                    __syncthreads();
                    evict_scan(sh);
#pragma unroll
                    for (int j = 0; j < kEvictItems; ++j) {
                        if (base + j * kEvictThreads >= n) break;
                        const uint32_t all = __ballot_sync(0xffffffffu, kept >> j & 1);
                        const uint32_t rank = at.equal + sh.count[j * kEvictWarps + warp] + __popc(all & ((1u << lane) - 1));
                        if (rank >= ties) kept &= ~(1u << j);
                    }
                    at.equal += sh.total;
                    __syncthreads();
                }
#pragma unroll
                for (int j = 0; j < kEvictItems; ++j) {
                    if (lane == 0) sh.count[j * kEvictWarps + warp] = 0;
                    if (base + j * kEvictThreads >= n) continue;
                    const int i = base + j * kEvictThreads + tid;
                    if (k[j] > key) kept |= 1u << j;
                    const bool stays = kept >> j & 1;
                    const bool moves = i < n && (i < many ? !stays : stays);
                    if (moves) move |= 1u << j;
                    const uint32_t all = __ballot_sync(0xffffffffu, moves);
                    const uint32_t low = __ballot_sync(0xffffffffu, moves && i < many);
                    if (lane == 0) sh.count[j * kEvictWarps + warp] = __popc(low) | __popc(all & ~low) << 16;
                }
                __syncthreads();
                evict_scan(sh);
#pragma unroll
                for (int j = 0; j < kEvictItems; ++j) {
                    if (base + j * kEvictThreads >= n) break;
                    const int i = base + j * kEvictThreads + tid;
                    const bool moves = move >> j & 1;
                    const uint32_t all = __ballot_sync(0xffffffffu, moves), low = __ballot_sync(0xffffffffu, moves && i < many);
                    const uint32_t count = sh.count[j * kEvictWarps + warp], before = (1u << lane) - 1;
                    if (!moves) continue;
                    const uint32_t x = (i < many ? at.holes + (count & 0xffff) + __popc(low & before)
                                                 : at.above + (count >> 16) + __popc(all & ~low & before)) -
                                       static_cast<uint32_t>(round);
                    if (x < kEvictMoves) (i < many ? sh.dst : sh.src)[x] = e.first + i;
                }
                at.holes += sh.total & 0xffff;
                at.above += sh.total >> 16;
                at.base += kEvictSpan;
                __syncthreads();
            }
            if (round == 0) fills = static_cast<int>(at.above);
        }
        const int total = fills + e.recent;
        for (int x = tid; x < kEvictMoves && round + x < total; x += kEvictThreads) {
            int src, dst;
            if (round + x < fills) {
                src = sh.src[x];
                dst = sh.dst[x];
            } else {
                src = tail + round + x - fills;
                dst = line + round + x - fills;
            }
            const int ls = kv.block.div(src), ld = kv.block.div(dst);
            sh.from[x] = (kv.at(table[ls], 0, src - ls * kv.block_size()) + head_at) * elem + column;
            sh.to[x] = (kv.at(table[ld], 0, dst - ld * kv.block_size()) + head_at) * elem + column;
            if (part == 0) mass_out[dst] = mass[src];
        }
        __syncthreads();
        const int here = total - round < kEvictMoves ? total - round : kEvictMoves;
        const int units = here * e.pieces;
        for (int which = 0; which < parts; ++which) {
            unsigned char* p = which ? static_cast<unsigned char*>(kv.v) : pool;
            for (int u0 = 0; u0 < units; u0 += kEvictThreads * kEvictAhead) {
                uint4 x[kEvictAhead];
                int64_t to[kEvictAhead];
#pragma unroll
                for (int j = 0; j < kEvictAhead; ++j) {
                    const int u = u0 + j * kEvictThreads + tid;
                    to[j] = -1;
                    if (u >= units) continue;
                    const int m = e.piece_div.div(u), c = (u - m * e.pieces) * 16;
                    x[j] = *reinterpret_cast<const uint4*>(p + sh.from[m] + c);
                    to[j] = sh.to[m] + c;
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < kEvictAhead; ++j)
                    if (to[j] >= 0) *reinterpret_cast<uint4*>(p + to[j]) = x[j];
            }
        }
        if (round + kEvictMoves >= total) break;
        __syncthreads();
    }
}

}  // namespace specv
