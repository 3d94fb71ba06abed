// cache_append.cuh -- keys and values of a pass into the paged cache, queries
// and keys turned by their rotary positions on the way.
//
// A token is a CTA: its position's angles are formed once in shared memory
// and serve every head.  Bound by memory for prompts and by a chain of three
// loads (length, block, row) for a few tokens; so a thread asks for its rows
// of q, k and v, whose places depend on nothing, before it looks at anything
// else (but the row count, where there is one: padding is not read), and what
// it gets is 16 bytes each: pieces of a head that turn together (j and
// j + rot / 2, or two neighbours).
//
// Measured (GB300, graph replays over sets of inputs of more than twice the L2;
// bytes counted once, of 6691 GB/s measured): 4 ragged prompts of up to 2048
// tokens, 32/8 heads of 128 in bf16, 26.1 us, 87%; 64 trees of 17 rows 7.7 us,
// 52% (5.7 with inputs in the L2); one token for 8 sequences 2.4 us (launch and
// the chain of loads).  Prompts issue an instruction in two of three cycles:
// rotation in packed pairs and angles that stay in registers took them from
// 51 us to 31, CTAs of half the threads (a token that waits holds less of the
// SM) to 28.6, leaving padding unread to 26.1 (in later sessions, with the same code,
// 29.9; trees 8.0).  One prompt of 32,768
// tokens takes 120 us, all of the copy rate; in blocks of 1 it takes 285,
// because every token looks at all blocks that its sequence writes to.
//
// Angles are formed in float64 (position * inv_freq passes 2^24 for far
// positions, where fp32 would lose the fraction of a turn), brought into
// [-pi, pi] there, and the sine and cosine are taken in fp32.
#pragma once
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace specv {

// Threads of a CTA: as many for a few tokens, half of them where the tokens
// are more than the SMs hold at once.  Prompts as above 28.6 us with 192, 26.1
// with 96 (64: 26.4), trees 8.9 and 7.7, one token for 8 sequences 2.4 and 2.7.
constexpr int kAppendFew = 192, kAppendMany = 96;
constexpr int kAppendResident = 960;  // threads of an SM
constexpr int kAppendHeads = 2;  // whose pieces a thread has in flight

// How the pairs lie: pieces apart, neighbours in a piece, or (where rot does
// not fill pieces) by values.
enum AppendMode { kApart = 0, kNeighbours = 1, kValues = 2 };

struct AppendArgs {
    KvView kv;
    const void *q, *k, *v;
    void* q_out;
    int64_t q_stride, k_stride, v_stride;
    const float* inv_freq;
    const int32_t* parents;
    const int32_t* row_counts;
    int32_t* row_status;
    int q_heads, rot, interleaved;
    FastDiv rows;   // of a sequence
    FastDiv units;  // pairs of pieces of a head
};

// cos and sin of the angle pos * f.
__device__ __forceinline__ float2 append_turn(int pos, float f) {
    const double a = static_cast<double>(pos) * static_cast<double>(f);
    const double two_pi = 6.283185307179586476925286766559;
    const double turns = rint(a * 0.15915494309189533576888376337251);
    float s, c;
    sincosf(static_cast<float>(fma(-turns, two_pi, a)), &s, &c);
    return make_float2(c, s);
}

template <typename T>
__device__ __forceinline__ void append_pair(T& x0, T& x1, float c, float s) {
    const float a = KvType<T>::load(x0), b = KvType<T>::load(x1);
    x0 = KvType<T>::store(a * c - b * s);
    x1 = KvType<T>::store(a * s + b * c);
}

// Pairs x[e], y[e] of two pieces, two at a time in packed arithmetic.
__device__ __forceinline__ void append_apart(f2& x, f2& y, f2 c, f2 s) {
    const f2 a = x, b = y;
    x = sub2(mul2(a, c), mul2(b, s));
    y = fma2(a, s, mul2(b, c));
}
__device__ __forceinline__ void append_pieces(KvVec<float>& x, KvVec<float>& y, const float* c, const float* s) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        f2 a = pack2(x.x[e], x.x[e + 1]), b = pack2(y.x[e], y.x[e + 1]);
        append_apart(a, b, pack2(c[e], c[e + 1]), pack2(s[e], s[e + 1]));
        unpack2(a, x.x[e], x.x[e + 1]);
        unpack2(b, y.x[e], y.x[e + 1]);
    }
}
__device__ __forceinline__ void append_pieces(KvVec<__nv_bfloat16>& x, KvVec<__nv_bfloat16>& y, const float* c,
                                              const float* s) {
    uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
    uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f2 a = pack2(bf16_lo(xw[e]), bf16_hi(xw[e])), b = pack2(bf16_lo(yw[e]), bf16_hi(yw[e]));
        append_apart(a, b, pack2(c[2 * e], c[2 * e + 1]), pack2(s[2 * e], s[2 * e + 1]));
        float lo, hi;
        unpack2(a, lo, hi);
        xw[e] = kv_pack_bf16(lo, hi);
        unpack2(b, lo, hi);
        yw[e] = kv_pack_bf16(lo, hi);
    }
}

// A thread has the same two pieces (a unit) of every hstep-th head, so that it
// keeps the angles that turn them.  Heads are counted through q, k and v.
template <typename T, int MODE, int THREADS>
__global__ void __launch_bounds__(THREADS, kAppendResident / THREADS) cache_append_kernel(const AppendArgs a) {
    constexpr int kVec = KvType<T>::kVec;
    using Vec = KvVec<T>;
    __shared__ __align__(16) float s_cos[128], s_sin[128];
    const int rows = static_cast<int>(a.rows.d);
    const int b = a.rows.div(blockIdx.x), r = blockIdx.x - b * rows;
    const int tid = threadIdx.x;
    const KvView& kv = a.kv;
    const int turning = a.q_heads + kv.heads, heads = turning + kv.heads;
    const int per = static_cast<int>(a.units.d), hstep = THREADS / per;
    const int h0 = a.units.div(tid), u = tid - h0 * per;
    const int half = a.rot / 2;
    // the unit's pieces of a head that turns, and of a value's
    const bool apart = MODE == kApart && u < half / kVec;
    const int x0 = apart ? u * kVec : MODE == kApart ? a.rot + 2 * (u * kVec - half) : 2 * u * kVec;
    const int y0 = apart ? x0 + half : x0 + kVec;
    // the token's queries, keys and values, at the first head as heads are counted
    const int64_t token = blockIdx.x;
    const T* q = static_cast<const T*>(a.q) + token * a.q_stride;
    const T* k = static_cast<const T*>(a.k) + token * a.k_stride - a.q_heads * kv.dim;
    const T* v = static_cast<const T*>(a.v) + token * a.v_stride - turning * kv.dim;
    T* q_out = static_cast<T*>(a.q_out) + token * a.q_heads * kv.dim;
    Vec x[kAppendHeads], y[kAppendHeads];
    auto load = [&](int h, int j) {
        if (h >= heads) return;
        const T* p = (h < a.q_heads ? q : h < turning ? k : v) + h * kv.dim;
        x[j] = *reinterpret_cast<const Vec*>(p + (h < turning ? x0 : 2 * u * kVec));
        y[j] = *reinterpret_cast<const Vec*>(p + (h < turning ? y0 : 2 * u * kVec + kVec));
    };
    auto load_all = [&](int h1) {
        if (h0 >= hstep) return;
#pragma unroll
        for (int j = 0; j < kAppendHeads; ++j) load(h1 + j * hstep, j);
    };
    // (where rows are counted, a row that is padding is not read)
    const int counted = a.row_counts ? a.row_counts[b] : rows;
    if (MODE != kValues && r < counted) load_all(h0);
    // the token's sequence: its length, its tree, the blocks it writes to.  Every token of a sequence looks at all of
    // them, so that of a refused sequence nothing is written
    const int len = kv.lens[b];
    const int count = a.row_counts || len != 0 ? counted : 0;
    const int base = len - count, slot = base + r;
    const int32_t* table = kv.tables + static_cast<int64_t>(b) * kv.max_blocks;
    int status = 0, blk = 0;
    if (count < 0 || count > rows || len < 0 || (count > 0 && (len < count || !kv.fits(len)))) status = KV_LENGTH;
    if (status == 0 && count > 0) {
        bool parent_bad = false, block_bad = false;
        int depth = r;
        if (a.parents) {
            uint32_t anc;
            int d;
            parent_bad = !warp_tree(a.parents + static_cast<int64_t>(b) * (rows - 1), count, tid & 31, anc, d);
            depth = __shfl_sync(0xffffffffu, d, r);
        }
        if (r < count) blk = table[kv.block.div(slot)];
        for (int i = kv.block.div(base) + tid, last = kv.block.div(len - 1); i <= last; i += THREADS)
            block_bad |= !kv.valid(table[i]);
        for (int j = tid; j < half; j += THREADS) {
            const float2 cs = append_turn(base + depth, a.inv_freq[j]);
            s_cos[j] = cs.x;
            s_sin[j] = cs.y;
        }
        if (__syncthreads_or(parent_bad || block_bad))
            status = (__syncthreads_or(parent_bad) ? KV_PARENT : 0) | (__syncthreads_or(block_bad) ? KV_BLOCK : 0);
    }
    if (r == 0 && tid == 0 && a.row_status) a.row_status[b] = status;
    if (status != 0 || r >= count) {
        if (a.q)
            for (int i = tid; i < a.q_heads * per * 2; i += THREADS)
                reinterpret_cast<uint4*>(q_out)[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int64_t at = kv.at(blk, 0, slot - kv.block.div(slot) * kv.block_size());
    const int64_t next = static_cast<int64_t>(kv.block_size()) * kv.dim;  // from a head of a block to the next
    T* k_out = static_cast<T*>(kv.k) + at;
    T* v_out = static_cast<T*>(kv.v) + at;
    if constexpr (MODE == kValues) {
        const int pairs = kv.dim / 2;  // of a head: the turning ones, then the rest by twos
        for (int i = tid; i < heads * pairs; i += THREADS) {
            const int h = i / pairs, j = i - h * pairs;
            const T* p = (h < a.q_heads ? q : h < turning ? k : v) + h * kv.dim;
            T* to = h < a.q_heads ? q_out + h * kv.dim
                    : h < turning ? k_out + (h - a.q_heads) * next
                                  : v_out + (h - turning) * next;
            const bool turns = h < turning && j < half, far = turns && !a.interleaved;
            const int d0 = far ? j : 2 * j, d1 = far ? j + half : 2 * j + 1;
            T e0 = p[d0], e1 = p[d1];
            if (turns) append_pair(e0, e1, s_cos[j], s_sin[j]);
            to[d0] = e0;
            to[d1] = e1;
        }
    } else {
        if (h0 >= hstep) return;
        // angles of the unit: of pairs x[e], y[e], or of the neighbours in x and then in y
        const int first = MODE == kApart ? x0 : x0 / 2;
        const bool turns = MODE == kApart ? apart : x0 < a.rot;
        const bool both = MODE == kApart || y0 < a.rot;  // (neighbours: whether the second piece turns too)
        float c[kVec], s[kVec];
        if (turns) {
#pragma unroll
            for (int e = 0; e < kVec; e += 4) {
                *reinterpret_cast<float4*>(c + e) = *reinterpret_cast<const float4*>(s_cos + first + e);
                *reinterpret_cast<float4*>(s + e) = *reinterpret_cast<const float4*>(s_sin + first + e);
            }
        }
        for (int h1 = h0; h1 < heads; h1 += kAppendHeads * hstep) {
            if (h1 != h0) load_all(h1);
#pragma unroll
            for (int j = 0; j < kAppendHeads; ++j) {
                const int h = h1 + j * hstep;
                if (h >= heads) continue;
                if (h < turning && turns) {
                    if constexpr (MODE == kApart) {
                        append_pieces(x[j], y[j], c, s);
                    } else {
#pragma unroll
                        for (int e = 0; e < kVec; e += 2) append_pair(x[j].x[e], x[j].x[e + 1], c[e / 2], s[e / 2]);
                        if (both) {
#pragma unroll
                            for (int e = 0; e < kVec; e += 2)
                                append_pair(y[j].x[e], y[j].x[e + 1], c[(kVec + e) / 2], s[(kVec + e) / 2]);
                        }
                    }
                }
                T* to = h < a.q_heads ? q_out + h * kv.dim
                        : h < turning ? k_out + (h - a.q_heads) * next
                                      : v_out + (h - turning) * next;
                *reinterpret_cast<Vec*>(to + (h < turning ? x0 : 2 * u * kVec)) = x[j];
                *reinterpret_cast<Vec*>(to + (h < turning ? y0 : 2 * u * kVec + kVec)) = y[j];
            }
        }
    }
}

}  // namespace specv
