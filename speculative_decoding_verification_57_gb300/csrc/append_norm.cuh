// append_norm.cuh -- the append of cache_append.cuh for models that norm the
// heads of queries and keys, and for positions on several axes: a head x
// becomes x * rsqrt(mean(x^2) + eps) * (weight + weight_add), and its pairs
// turn by position * inv_freq as there, the position being that of the pair's
// axis (positions[b, r, axis]) or, with one axis, base + depth(r) + offset[b].
// Everything between the loads and the one rounding at the end is fp32 (the
// angle float64); a head whose squares leave that type's range, or vanish in it,
// is summed once more, scaled by a power of two.
//
// Layout, loads ahead of the length and the rest as in cache_append.cuh.  A
// head belongs to a group of 1, 2, 4, .. 32 neighbouring lanes, the least that
// hold its pieces, so that its sum of squares is added up by shuffles; lanes
// behind the head's pieces (heads of 96: two of eight) are idle.  A thread has
// the same two pieces of every head it works on: the products of their weights
// with their sines and cosines stay in its registers, for queries and then
// for keys, so that a norm costs a head eight multiply-adds, the shuffles and
// eight products more than the turn.
//
// Measured (GB300, graph replays over sets of inputs beyond the L2; 32/8 heads of
// 128 in bf16): one token for 8 sequences 3.7 us (2.5 without norms), 64 trees of 17
// rows 10.3 us (8.0), 4 ragged prompts of up to 2048 tokens with images on three
// axes 39.7 us, 56% of 6803 GB/s (with one axis 37.5, without norms 35.4, with neither
// 34.4, the plain append 29.9); fp32 57.4 us, 77%.  Bound by instructions and the chain
// of loads together: 1.98 of 4 instructions a cycle with 21 warps an SM.  No one part
// of it weighs: angles, shuffles, weights, stores and the look at the blocks are 1 to
// 4 us each.  Part of the chain stands without need, left for another time: positions,
// angles and weights depend on neither length nor block, and are asked for behind both.
#pragma once
#include "cache_append.cuh"

namespace specv {

struct AppendNormArgs {
    AppendArgs a;
    const void *q_weight, *k_weight;  // [head_dim] of the cache's type; NULL: not normed
    const int32_t* positions;         // [B, rows, axes]; NULL: base + depth + offset
    const int32_t* offsets;           // [B]; NULL: 0
    float eps, weight_add, inv_dim;
    int axes;
    int group_log;  // lanes of a head, their base-2 logarithm
    uint8_t axis[128];  // of each pair
};

// cos and sin of the angle pos * f, formed as append_turn forms it.
__device__ __forceinline__ float2 append_turn_at(double pos, float f) {
    const double a = pos * static_cast<double>(f);
    const double two_pi = 6.283185307179586476925286766559;
    const double turns = rint(a * 0.15915494309189533576888376337251);
    float s, c;
    sincosf(static_cast<float>(fma(-turns, two_pi, a)), &s, &c);
    return make_float2(c, s);
}

// Whether a mean of squares (and eps) lost nothing to fp32's range: squares below 2^-126 lose bits, of which this has 35
// to spare, and a sum beyond the type is infinite.  Where not, the head is scaled by a power of two first.
__device__ __forceinline__ bool append_mean_fits(float mean) { return mean >= 0x1p-90f && mean < INFINITY; }

// The power of two that brings `top`, a head's largest magnitude or the root of eps, to 1..2 (ends of the type: near them).
__device__ __forceinline__ float append_scale(float top) {
    const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
    return __uint_as_float((254 - e) << 23);
}

// 16 bytes as floats, two at a time, and back.
template <typename T>
__device__ __forceinline__ void append_open(const KvVec<T>& x, f2 (&f)[KvType<T>::kVec / 2]) {
    if constexpr (sizeof(T) == 2) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = pack2(bf16_lo(w[e]), bf16_hi(w[e]));
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) f[e] = pack2(x.x[2 * e], x.x[2 * e + 1]);
    }
}
template <typename T>
__device__ __forceinline__ void append_close(const f2 (&f)[KvType<T>::kVec / 2], KvVec<T>& x) {
#pragma unroll
    for (int e = 0; e < KvType<T>::kVec / 2; ++e) {
        float lo, hi;
        unpack2(f[e], lo, hi);
        if constexpr (sizeof(T) == 2) {
            reinterpret_cast<uint32_t*>(&x)[e] = kv_pack_bf16(lo, hi);
        } else {
            x.x[2 * e] = lo;
            x.x[2 * e + 1] = hi;
        }
    }
}

// Neighbours f[e] by (their weights times) the cosine, c[e], and the sine, s[e], of the pair.
template <int N>
__device__ __forceinline__ void append_neighbours(f2 (&f)[N], const f2 (&c)[N], const f2 (&s)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        float x, y, c0, c1, s0, s1;
        unpack2(f[e], x, y);
        unpack2(c[e], c0, c1);
        unpack2(s[e], s0, s1);
        f[e] = pack2(x * c0 - y * s1, x * s0 + y * c1);
    }
}

// Threads of an SM: more registers each than a plain append's need (576: trees 14.0 us, prompts 45.0; 768: 10.9 and 42.8;
// 960: 11.8 and 41.8).
// Tokens get the many threads of kAppendFew as long as the SMs hold all of them at once, three an SM (trees of 8 rows,
// 32/8 heads of 128 in bf16: 456 tokens 6.95 us; 464 in two turns 10.2, with the threads of kAppendMany 8.4; 760 11.6 and 9.5).
constexpr int kNormResident = 672;

template <typename T, int MODE, int THREADS>
__global__ void __launch_bounds__(THREADS, kNormResident / THREADS)
cache_append_norm_kernel(const __grid_constant__ AppendNormArgs n) {
    constexpr int kVec = KvType<T>::kVec, kTwos = kVec / 2;
    using Vec = KvVec<T>;
    __shared__ __align__(16) float s_cos[128], s_sin[128];
    __shared__ float s_head[MODE == kValues ? THREADS / 32 : 1][MODE == kValues ? 256 : 1];
    const AppendArgs& a = n.a;
    const int rows = static_cast<int>(a.rows.d);
    const int b = a.rows.div(blockIdx.x), r = blockIdx.x - b * rows;
    const int tid = threadIdx.x, lane = tid & 31;
    const KvView& kv = a.kv;
    const int turning = a.q_heads + kv.heads, heads = turning + kv.heads;
    const int per = static_cast<int>(a.units.d), hstep = THREADS >> n.group_log;
    const int h0 = tid >> n.group_log, u = tid - (h0 << n.group_log);
    const bool piece = u < per;  // the lane has pieces of its head
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
    auto load_all = [&](int h1) {
#pragma unroll
        for (int j = 0; j < kAppendHeads; ++j) {
            const int h = h1 + h0 + j * hstep;
            if (!piece || h >= heads) continue;
            const T* p = (h < a.q_heads ? q : h < turning ? k : v) + h * kv.dim;
            x[j] = *reinterpret_cast<const Vec*>(p + (h < turning ? x0 : 2 * u * kVec));
            y[j] = *reinterpret_cast<const Vec*>(p + (h < turning ? y0 : 2 * u * kVec + kVec));
        }
    };
    // (where rows are counted, a row that is padding is not read)
    const int counted = a.row_counts ? a.row_counts[b] : rows;
    if (MODE != kValues && r < counted) load_all(0);
    // the token's sequence, as in cache_append_kernel
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
            parent_bad = !warp_tree(a.parents + static_cast<int64_t>(b) * (rows - 1), count, lane, anc, d);
            depth = __shfl_sync(0xffffffffu, d, r);
        }
        if (r < count) {
            blk = table[kv.block.div(slot)];
            const int64_t at = static_cast<int64_t>(base) + depth + (n.offsets ? n.offsets[b] : 0);
            for (int j = tid; j < half; j += THREADS) {
                const double pos = n.positions ? static_cast<double>(n.positions[token * n.axes + n.axis[j]])
                                               : static_cast<double>(at);
                const float2 cs = append_turn_at(pos, a.inv_freq[j]);
                s_cos[j] = cs.x;
                s_sin[j] = cs.y;
            }
        }
        const int first_block = kv.block.div(base), many = kv.block.div(len - 1) - first_block + 1;
#pragma unroll 2
        for (int i = tid; i < many; i += THREADS)
            block_bad |= static_cast<uint32_t>(table[first_block + i]) >= static_cast<uint32_t>(kv.blocks);
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
        // a head a warp, through shared memory: pairs that do not fill pieces
        float* head = s_head[tid >> 5];
        for (int h = tid >> 5; h < heads; h += THREADS / 32) {
            const T* p = (h < a.q_heads ? q : h < turning ? k : v) + h * kv.dim;
            const bool normed = h < a.q_heads ? n.q_weight != nullptr : h < turning && n.k_weight;
            float sum = 0.0f;
            for (int d = lane; d < kv.dim; d += 32) {
                const float f = KvType<T>::load(p[d]);
                head[d] = f;
                sum = fmaf(f, f, sum);
            }
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            __syncwarp();
            float mean = fmaf(sum, n.inv_dim, n.eps);
            if (normed && !append_mean_fits(mean)) {  // (the whole warp: it has the head)
                float top = sqrtf(n.eps);
                for (int d = lane; d < kv.dim; d += 32) top = fmaxf(top, fabsf(head[d]));
                for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float s = append_scale(top);
                sum = 0.0f;
                for (int d = lane; d < kv.dim; d += 32) {
                    head[d] *= s;
                    sum = fmaf(head[d], head[d], sum);
                }
                for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                __syncwarp();
                mean = fmaf(sum, n.inv_dim, n.eps * s * s);
            }
            const float inv = normed ? rsqrtf(mean) : 1.0f;
            const T* w = static_cast<const T*>(h < a.q_heads ? n.q_weight : n.k_weight);
            T* to = h < a.q_heads ? q_out + h * kv.dim
                    : h < turning ? k_out + (h - a.q_heads) * next
                                  : v_out + (h - turning) * next;
            for (int j = lane; j < kv.dim / 2; j += 32) {  // the turning pairs, then the rest by twos
                const bool turns = h < turning && j < half, far = turns && !a.interleaved;
                const int d0 = far ? j : 2 * j, d1 = far ? j + half : 2 * j + 1;
                float e0 = head[d0], e1 = head[d1];
                if (normed) {
                    e0 *= inv * (KvType<T>::load(w[d0]) + n.weight_add);
                    e1 *= inv * (KvType<T>::load(w[d1]) + n.weight_add);
                }
                if (turns) {
                    const float c = s_cos[j], s = s_sin[j], f = e0;
                    e0 = f * c - e1 * s;
                    e1 = f * s + e1 * c;
                }
                to[d0] = KvType<T>::store(e0);
                to[d1] = KvType<T>::store(e1);
            }
            __syncwarp();
        }
    } else {
        // angles of the unit: of pairs x[e], y[e], or of the neighbours in x and then in y
        const int first = MODE == kApart ? x0 : x0 / 2;
        const bool turns = piece && (MODE == kApart ? apart : x0 < a.rot);
        const bool both = MODE == kApart || y0 < a.rot;  // (neighbours: whether the second piece turns too)
        // the pieces' weights, times cosines and sines where they turn: of x with cos and sin of its pairs, of y alike
        f2 cx[kTwos], sx[kTwos], cy[kTwos], sy[kTwos];
        auto coefficients = [&](const T* w) {
#pragma unroll
            for (int e = 0; e < kTwos; ++e) cx[e] = cy[e] = pack2(1.0f, 1.0f);
            if (w) {
                const f2 add = pack2(n.weight_add, n.weight_add);
                append_open<T>(*reinterpret_cast<const Vec*>(w + x0), cx);
                append_open<T>(*reinterpret_cast<const Vec*>(w + y0), cy);
#pragma unroll
                for (int e = 0; e < kTwos; ++e) {
                    cx[e] = add2(cx[e], add);
                    cy[e] = add2(cy[e], add);
                }
            }
            if (!turns) return;
            if constexpr (MODE == kApart) {
#pragma unroll
                for (int e = 0; e < kTwos; e += 2) {
                    const float4 c = *reinterpret_cast<const float4*>(s_cos + first + 2 * e);
                    const float4 s = *reinterpret_cast<const float4*>(s_sin + first + 2 * e);
                    const f2 c2[2] = {pack2(c.x, c.y), pack2(c.z, c.w)}, s2[2] = {pack2(s.x, s.y), pack2(s.z, s.w)};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        sx[e + k] = mul2(cx[e + k], s2[k]);
                        cx[e + k] = mul2(cx[e + k], c2[k]);
                        sy[e + k] = mul2(cy[e + k], s2[k]);
                        cy[e + k] = mul2(cy[e + k], c2[k]);
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < kTwos; ++e) {
                    const float c = s_cos[first + e], s = s_sin[first + e];
                    sx[e] = mul2(cx[e], pack2(s, s));
                    cx[e] = mul2(cx[e], pack2(c, c));
                    if (both) {
                        const float c1 = s_cos[first + kTwos + e], s1 = s_sin[first + kTwos + e];
                        sy[e] = mul2(cy[e], pack2(s1, s1));
                        cy[e] = mul2(cy[e], pack2(c1, c1));
                    }
                }
            }
        };
        // the warp's first head: those from `turning` on are values (told by a vote a head instead, trees took 10.7 us for
        // 10.3, image prompts 40.3 for 39.2)
        const int warp0 = __shfl_sync(0xffffffffu, h0, 0);
        const bool norms = n.q_weight || n.k_weight;
        int kind = -1;  // whose they are: 0 queries', 1 keys'
        auto has_norm = [&](int h) { return piece && (h < a.q_heads ? n.q_weight != nullptr : h < turning && n.k_weight); };
        auto squares = [&](const f2 (&fx)[kTwos], const f2 (&fy)[kTwos]) {
            f2 sum = pack2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < kTwos; ++e) sum = fma2(fx[e], fx[e], fma2(fy[e], fy[e], sum));
            float lo, hi;
            unpack2(sum, lo, hi);
            return lo + hi;
        };
        // mean of a head's squares and eps, by its lanes
        auto mean_of = [&](bool normed, const f2 (&fx)[kTwos], const f2 (&fy)[kTwos], float eps) {
            float all = normed ? squares(fx, fy) : 0.0f;
#pragma unroll
            for (int step = 4; step >= 0; --step)
                if (step < n.group_log) all += __shfl_xor_sync(0xffffffffu, all, 1 << step);
            return fmaf(all, n.inv_dim, eps);
        };
        // a query's or key's pieces, normed and turned
        auto turn = [&](int h, f2 (&fx)[kTwos], f2 (&fy)[kTwos], float inv, Vec& xo, Vec& yo) {
            if (kind != (h < a.q_heads ? 0 : 1)) {
                kind = h < a.q_heads ? 0 : 1;
                coefficients(static_cast<const T*>(kind ? n.k_weight : n.q_weight));
            }
            const f2 inv2 = pack2(inv, inv);
            if (!turns) {
#pragma unroll
                for (int e = 0; e < kTwos; ++e) {
                    fx[e] = mul2(fx[e], mul2(inv2, cx[e]));
                    fy[e] = mul2(fy[e], mul2(inv2, cy[e]));
                }
            } else {
                if constexpr (MODE == kApart) {
#pragma unroll
                    for (int e = 0; e < kTwos; ++e) {
                        const f2 v = fx[e], w = fy[e];
                        fx[e] = sub2(mul2(v, cx[e]), mul2(w, sy[e]));
                        fy[e] = fma2(v, sx[e], mul2(w, cy[e]));
                    }
                } else {
                    append_neighbours<kTwos>(fx, cx, sx);
                    if (both) append_neighbours<kTwos>(fy, cy, sy);
                }
#pragma unroll
                for (int e = 0; e < kTwos; ++e) {
                    fx[e] = mul2(fx[e], inv2);
                    fy[e] = MODE == kApart || both ? mul2(fy[e], inv2) : mul2(fy[e], mul2(inv2, cy[e]));
                }
            }
            append_close<T>(fx, xo);
            append_close<T>(fy, yo);
        };
        auto store = [&](int h, const Vec& xo, const Vec& yo) {
            T* to = h < a.q_heads ? q_out + h * kv.dim
                    : h < turning ? k_out + (h - a.q_heads) * next
                                  : v_out + (h - turning) * next;
            *reinterpret_cast<Vec*>(to + (h < turning ? x0 : 2 * u * kVec)) = xo;
            *reinterpret_cast<Vec*>(to + (h < turning ? y0 : 2 * u * kVec + kVec)) = yo;
        };
        for (int h1 = 0; h1 < heads; h1 += kAppendHeads * hstep) {
            if (h1 > 0) load_all(h1);
#pragma unroll
            for (int j = 0; j < kAppendHeads; ++j) {
                const int h = h1 + h0 + j * hstep;
                const bool mine = piece && h < heads, normed = has_norm(h);
                f2 fx[kTwos], fy[kTwos];
                float inv = 1.0f;
                if (mine && h < turning) {
                    append_open<T>(x[j], fx);
                    append_open<T>(y[j], fy);
                }
                if (norms && h1 + warp0 + j * hstep < turning) {
                    float mean = mean_of(normed, fx, fy, n.eps);
                    const bool far = normed && !append_mean_fits(mean);
                    if (__any_sync(0xffffffffu, far)) {  // once more, scaled
                        float top = sqrtf(n.eps);
                        if (normed) {
#pragma unroll
                            for (int e = 0; e < kTwos; ++e) {
                                float p0, p1, r0, r1;
                                unpack2(fx[e], p0, p1);
                                unpack2(fy[e], r0, r1);
                                top = fmaxf(fmaxf(fmaxf(top, fabsf(p0)), fmaxf(fabsf(p1), fabsf(r0))), fabsf(r1));
                            }
                        }
#pragma unroll 1
                        for (int step = 0; step < n.group_log; ++step)
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1 << step));
                        const float s = far ? append_scale(top) : 1.0f;
                        float all = 0.0f;
                        if (normed) {
#pragma unroll
                            for (int e = 0; e < kTwos; ++e) {
                                fx[e] = mul2(fx[e], pack2(s, s));
                                fy[e] = mul2(fy[e], pack2(s, s));
                            }
                            all = squares(fx, fy);
                        }
#pragma unroll 1
                        for (int step = 0; step < n.group_log; ++step) all += __shfl_xor_sync(0xffffffffu, all, 1 << step);
                        mean = fmaf(all, n.inv_dim, n.eps * s * s);
                    }
                    if (normed) inv = rsqrtf(mean);
                }
                if (!mine) continue;
                if (h < turning) turn(h, fx, fy, inv, x[j], y[j]);
                store(h, x[j], y[j]);
            }
        }
    }
}

}  // namespace specv
