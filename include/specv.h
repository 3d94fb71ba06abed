/*
 * specv.h -- C ABI of the batched speculative-decoding verify step on one
 * GB300 (sm_103a).
 *
 * For every sequence b of a batch the library scores k draft tokens against
 * the target model's k+1 output distributions and emits between 1 and k+1
 * tokens whose distribution is exactly the target's:
 *
 *   1. p_i = softmax(target_logits[b,i,:] / T_b) at each position i = 0..k
 *      ("Speculative decoding." lesson, "First: what an output distribution
 *      is": softmax of the logits, temperature divides them first);
 *   2. draft token x_i is kept iff U[b,i,0] < min(1, p_i(x_i) / q_i(x_i)),
 *      q_i(x_i) clamped below at 1e-12 ("LLM Inference & Speculative
 *      Decoding: From Roofline Physics to Lossless Acceleration", s.2,
 *      acceptance rule and its PyTorch verification step);
 *   3. the walk stops at the first rejected position j ("Speculative
 *      Decoding: Mathematical Foundations, ...", "The Modified Rejection
 *      Sampling Algorithm": later drafts are discarded);
 *   4. at j < k one token is drawn from max(0, p_j - q_j) normalised, by
 *      inverse CDF with U[b,j,1]; if all k drafts are kept, the bonus token is
 *      drawn from p_k with U[b,k,1] (same sources, residual distribution and
 *      bonus token).  If the residual has zero mass, p_j is sampled instead
 *      ("Speculative Decoding: Draft, Verify, Accept", demo script part B).
 *   Rows with T_b == 0 use the greedy rule: keep x_i while it equals
 *   argmax p_i (lowest index on ties), emit the argmax at the first mismatch
 *   or at position k ("LLM Inference & Speculative Decoding ...", s.4 fix for
 *   T -> 0; "Speculative Decoding: Mathematical Foundations, ...", "Greedy
 *   Decoding Equivalence").
 *
 * Inverse CDF: the emitted token is the smallest v (vocabulary order) with
 *   u * W < w(0) + ... + w(v), W the total weight ("Speculative decoding."
 *   lesson: lay the probabilities end to end and take the slice u lands in).
 *
 * Layouts (all row-major, contiguous, device memory unless stated):
 *   target_logits [B, k+1, V]  bf16 (SPECV_BF16) or fp32 (SPECV_F32)
 *   draft_probs   [B, k, V]    fp32, the distribution the drafts were drawn
 *                              from, used as given (never re-tempered); or
 *                              NULL for one-hot drafts (prompt lookup, n-gram
 *                              or greedy drafting: q is the point mass at the
 *                              draft token, so a draft is kept with
 *                              probability p(x) and a rejection samples p with
 *                              x removed -- "Speculative decoding." lesson,
 *                              "One guess (lookup)", "N-gram and prompt
 *                              lookup"; no page gives a separate call for it)
 *   draft_tokens  [B, k]       int32
 *   uniforms      [B, k+1, 2]  fp32 in [0,1); [b,i,0] drives the accept test
 *                              at i < k, [b,j,1] the residual/bonus draw at
 *                              the stop position j; [b,k,0] is unused
 *   temperature   [B]          fp32; 0 = greedy row; otherwise a finite
 *                              normal positive float
 *   num_accepted  [B]          int32 out, j in [0, k]; the row emits j+1 tokens
 *   out_tokens    [B, k+1]     int32 out: x_0..x_{j-1}, then the fixed or
 *                              bonus token at index j, then -1
 *   row_status    [B]          int32 out (nullable), bit mask:
 *                                1  non-finite logits at an examined position
 *                                   (a NaN or +inf, or all -inf; greedy rows:
 *                                   a NaN)
 *                                2  draft token outside [0, V)
 *                                4  uniform outside [0, 1)
 *                                8  temperature negative, NaN, infinite or
 *                                   subnormal
 *                               16  (information) residual mass was zero, the
 *                                   token was drawn from p_j
 *                               32  draft probability NaN, negative or
 *                                   infinite at an examined entry
 *                               64  an internal wait timed out (the result of
 *                                   this row is not valid)
 *                              128  (rollback, KV cache compaction) an
 *                                   accepted count out of range
 *                              256  (rollback) no room in the free list
 *                              512  (trees) a parent index
 *                                   outside [-1, node)
 *                             1024  (top-k / top-p verification) top_k
 *                                   outside [1, 4096] or top_p outside (0, 1]
 *                             2048  (KV cache) a sequence length or row count
 *                                   that does not fit (see specv_kv_cache)
 *                             4096  (KV cache) a block table entry in use
 *                                   outside the pool
 *                             8192  (KV cache compaction) a path that is not
 *                                   strictly increasing inside [0, M)
 *                              The walk checks position 0, 1, ... in order and
 *                              stops at the first position with an error; a
 *                              row with any of the bits 1, 2, 4, 8, 32, 64, 512, 1024 set
 *                              reports num_accepted = 0 and out_tokens = -1.
 *
 * Ownership and execution: the caller owns every buffer.  Calls are
 * asynchronous on the given CUDA stream (a cudaStream_t passed as void*;
 * NULL is the legacy default stream) and allocate nothing; argument errors
 * are reported synchronously before anything is launched.  A handle may be
 * used from one host thread at a time.  Pointers need no particular
 * alignment; sizes are limited by the handle (batch <= max_batch,
 * 1 <= k <= max_k, V <= vocab).
 */
#ifndef SPECV_H
#define SPECV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct specv_ctx *specv_handle;

typedef enum {
    SPECV_OK = 0,
    SPECV_ERR_INVALID_ARGUMENT = 1, /* bad pointer, size or dtype; nothing launched */
    SPECV_ERR_UNSUPPORTED = 2,      /* device is not sm_103 or lacks a needed feature */
    SPECV_ERR_CUDA = 3,             /* a CUDA runtime call failed (see specv_last_cuda_error) */
    SPECV_ERR_TIMEOUT = 4           /* reserved: reported per row as row_status bit 64 */
} specv_status;

typedef enum { SPECV_F32 = 0, SPECV_BF16 = 1 } specv_dtype;

/* Optional intermediates, all device pointers, each nullable.  For greedy
 * rows row_sumexp, p_at_draft, q_at_draft and residual_mass are 0. */
typedef struct {
    float *p_at_draft;    /* [B, k]   p_i(x_i) (0 if x_i is out of range) */
    float *q_at_draft;    /* [B, k]   q_i(x_i) as read, 1 for one-hot drafts (0 if out of range) */
    float *row_max;       /* [B, k+1] max_v logits[b,i,v] */
    float *row_sumexp;    /* [B, k+1] sum_v exp((logits[b,i,v] - row_max) / T) */
    float *residual_mass; /* [B]      sum_v max(0, p_j(v) - q_j(v)) at a rejected
                                      position (1 - p_j(x_j) for one-hot drafts),
                                      else 0 */
} specv_debug;

/* Create a handle on CUDA device `device` for batches up to max_batch rows,
 * 1 <= k <= max_k (1 <= max_k <= 31: positions 0..k fit one warp) and
 * vocabularies up to `vocab` entries (1 <= vocab <= 262144: at most 16 CTAs
 * of 16384 entries a position).  Other values: SPECV_ERR_INVALID_ARGUMENT.
 * Queries the device; allocates no device memory.  Returns
 * SPECV_ERR_UNSUPPORTED if the device is not compute capability 10.3.
 * Two environment variables, read at every call, override the launch plan
 * (for tests and tuning; the results do not depend on them):
 * SPECV_CLUSTER=C (V > 2048: C CTAs per row, from the fewest the slice limit
 * allows up to 16) and SPECV_SMALLV=row|warp (V <= 2048: one CTA of eight
 * warps per row, or one warp per row; by default the first while the batch
 * is at most twice the SM count). */
specv_status specv_create(specv_handle *out, int device, int max_batch, int max_k, int64_t vocab);

/* Sampled verification (rows with temperature 0 take the greedy rule).
 * target_logits: dtype logits_dtype; every other pointer as in the layout
 * table above; dbg may be NULL.  V = vocabulary size of this call. */
specv_status specv_verify_sample(specv_handle h, specv_dtype logits_dtype, const void *target_logits,
                                 const float *draft_probs, const int32_t *draft_tokens,
                                 const float *uniforms, const float *temperature, int batch, int k,
                                 int64_t V, int32_t *num_accepted, int32_t *out_tokens,
                                 int32_t *row_status, const specv_debug *dbg, void *stream);

/* Sampled verification with top-k / top-p applied to each target row before
 * the rule ("Speculative decoding." lesson, "Why the output is exactly p":
 * temperature, top-k and top-p have to be applied to p before the rule, and
 * to q before drafting -- q is used as given).  The pages name the filters
 * without defining them; the readings here:
 *   top_k [B] int32, 1..4096: keep the top_k largest logits (all V if
 *         top_k >= V), the lower index first among equal logits;
 *   top_p [B] fp32, (0, 1]: within those, in the same order, keep the
 *         shortest prefix whose mass (renormalised over the top_k) reaches
 *         top_p (at least one entry; 1 keeps all top_k).
 * p' = exp((l - max) / T) on the kept set, renormalised; the accept test,
 * the residual max(0, p' - q) and the bonus use p'.  The residual and the
 * bonus are drawn over the kept set in vocabulary order; q is read (and
 * checked, bit 32) only there and at the draft tokens.  draft_probs may be
 * NULL (one-hot drafts), device memory, or page-locked host memory, read in
 * place (pageable host memory: SPECV_ERR_INVALID_ARGUMENT).  A row whose
 * top_k or top_p is out of range gets row_status bit 1024 and emits
 * nothing.  Rows with temperature 0 take the greedy rule (the filters keep
 * the argmax).  Other arguments and bits as for specv_verify_sample; no
 * debug outputs.  Two launches on the stream: rows with top_k up to 64 (and
 * greedy or refused rows) take one thread-block cluster of min(k + 1, 8)
 * CTAs per row that keeps each position's best 64 in registers; rows with
 * top_k above 64 take a cluster of min(k + 1, 16) CTAs per row that selects
 * each position's kept set exactly by a radix select on the logits' keys. */
specv_status specv_verify_sample_filtered(specv_handle h, specv_dtype logits_dtype, const void *target_logits,
                                          const float *draft_probs, const int32_t *draft_tokens,
                                          const float *uniforms, const float *temperature, const int32_t *top_k,
                                          const float *top_p, int batch, int k, int64_t V, int32_t *num_accepted,
                                          int32_t *out_tokens, int32_t *row_status, void *stream);

/* Greedy verification of every row (no draft probabilities, uniforms or
 * temperatures): keep x_i while it equals the target argmax. */
specv_status specv_verify_greedy(specv_handle h, specv_dtype logits_dtype, const void *target_logits,
                                 const int32_t *draft_tokens, int batch, int k, int64_t V,
                                 int32_t *num_accepted, int32_t *out_tokens, int32_t *row_status,
                                 void *stream);

/* Greedy verification of draft trees ("LLM Inference & Speculative Decoding:
 * From Roofline Physics to Lossless Acceleration", s.3 "Multi-Draft Tree
 * Speculation"; "Speculative Decoding: Mathematical Foundations, ...",
 * "SpecInfer and Tree-Based Verification": the target scores every node in
 * one pass and the longest accepted path is kept).  Device pointers:
 *   target_logits [B, M+1, V]  row 0: the prediction after the prefix;
 *                              row 1+i: the prediction after node i
 *   tokens        [B, M]       int32, the draft token of each node
 *   parents       [B, M]       int32, parent node of each node, in [-1, i)
 *                              (-1: a child of the prefix)
 *   num_accepted  [B]          out: length of the kept path
 *   out_tokens    [B, M+1]     out: the path's tokens from the prefix down,
 *                              then the bonus (argmax after the path's last
 *                              node, or of row 0), -1 after
 *   path          [B, M]       out (nullable): the path's node indices, -1 after
 *   row_status    [B]          out (nullable): 0, or bits 1 (a NaN logit in
 *                              any row), 2 (a token outside [0, V)), 512 (a
 *                              parent outside [-1, i)); such rows emit nothing
 * A node is kept iff its parent is kept (the prefix always is) and its
 * token is the argmax (lowest index on ties) of its parent's row; the
 * deepest kept node wins, the lowest index among equally deep ones.  The
 * pages define the path only in words; this is the plain reading.  A chain
 * (parent i-1) gives exactly specv_verify_greedy.  1 <= M <= max_k. */
specv_status specv_verify_tree_greedy(specv_handle h, specv_dtype logits_dtype, const void *target_logits,
                                      const int32_t *tokens, const int32_t *parents, int batch, int M, int64_t V,
                                      int32_t *num_accepted, int32_t *out_tokens, int32_t *path,
                                      int32_t *row_status, void *stream);

/* Same as specv_verify_sample, but every pointer is HOST memory (pinned
 * memory gives the fastest copies).  The handle copies the inputs to device
 * buffers it owns (allocated on the first call, grown when a larger call
 * comes; this is the one call that may allocate), verifies, copies the three
 * outputs back and synchronises `stream` before returning.  draft_probs in
 * page-locked host memory (cudaHostAlloc / cudaHostRegister) is not copied:
 * the kernel reads in place the entries the rule needs (q at the draft
 * tokens and the stop rows), with plain loads; pageable draft_probs is
 * copied like the other inputs. */
specv_status specv_verify_sample_host(specv_handle h, specv_dtype logits_dtype, const void *target_logits,
                                      const float *draft_probs, const int32_t *draft_tokens,
                                      const float *uniforms, const float *temperature, int batch,
                                      int k, int64_t V, int32_t *num_accepted, int32_t *out_tokens,
                                      int32_t *row_status, void *stream);

/* Paged KV-cache bookkeeping after a verification ("LLM Inference &
 * Speculative Decoding: From Roofline Physics to Lossless Acceleration", s.1,
 * PagedKVCacheManager.rollback_to), all pointers device memory:
 *   num_accepted [B]               int32, as returned by a verify call
 *   seq_lens     [B]               int32 in/out: positions held in the cache,
 *                                  the last k of them the drafts; becomes
 *                                  seq_len - (k - num_accepted)
 *   block_tables [B, max_blocks]   int32 in/out: physical block of each
 *                                  logical block; popped entries become -1
 *   num_blocks   [B]               int32 in/out: blocks in use; becomes
 *                                  ceil(new seq_len / block_size)
 *   free_list    [free_capacity]   int32: freed blocks are appended
 *   free_count   [1]               int32 in/out: entries used in free_list
 *   row_status   [B]               int32 out (nullable): 0; 128 if the row's
 *                                  num_accepted is outside [0, k], its new
 *                                  length would be negative or num_blocks is
 *                                  outside [0, max_blocks] (the row is left
 *                                  as it is); 256 on every row if the free
 *                                  list has no room for all freed blocks
 *                                  (then nothing changes)
 * The result equals rolling the rows back one at a time in batch order,
 * each row's blocks popped last-first.  Asynchronous on `stream`; argument
 * errors are returned before launch (SPECV_ERR_INVALID_ARGUMENT, among them
 * free_capacity outside [0, INT32_MAX]: free_count is an int32). */
specv_status specv_rollback(specv_handle h, const int32_t *num_accepted, int batch, int k, int32_t *seq_lens,
                            int32_t *block_tables, int max_blocks, int32_t *num_blocks, int block_size,
                            int32_t *free_list, int64_t free_capacity, int32_t *free_count, int32_t *row_status,
                            void *stream);

/* A paged KV cache of one layer, as specv_rollback keeps it ("LLM Inference &
 * Speculative Decoding: From Roofline Physics to Lossless Acceleration", s.1,
 * PagedKVCacheManager: a pool of blocks [blocks, heads, block_size, head_dim]
 * for the keys, one for the values, and a block table per sequence).  Every
 * pointer is device memory:
 *   k, v          the two pools, element type dtype.  Inside a block
 *                 [kv_heads, block_size, head_dim] without gaps; block_stride
 *                 elements from one block to the next (the same in both), so
 *                 that a pool may be a slice of a larger tensor
 *   block_tables  [B, max_blocks] int32: block of each logical block
 *   seq_lens      [B] int32: positions held, the rows of the current pass the
 *                 last of them (position t is in block t / block_size of the
 *                 table, at t % block_size).  0: an idle sequence (padding of
 *                 a batch): nothing of it is read from the cache, its status
 *                 is 0, and what its rows in the calls' tensors hold (they
 *                 have to be readable all the same) has no effect
 * head_dim is a multiple of 16 from 16 to 256, block_size 1..65536, blocks at
 * most 2^31 - 1; k, v and the tensors of the calls below are 16-byte aligned,
 * and so is block_stride in bytes.  Sizes outside these, or a block_stride
 * below kv_heads * block_size * head_dim: SPECV_ERR_INVALID_ARGUMENT.
 * A sequence is refused, with its row_status saying why, if its length is
 * negative, below the rows of the pass (0 aside), above max_blocks *
 * block_size or above 2^31 - 513 (bit 2048), or if an entry of its table that the call needs is
 * outside [0, blocks) (bit 4096).
 * What a call writes is memory apart from what it reads, where its
 * description does not say otherwise. */
typedef struct {
    specv_dtype dtype;
    int kv_heads, head_dim, block_size, max_blocks;
    void *k, *v;
    int64_t blocks;
    int64_t block_stride;
    const int32_t *block_tables;
    const int32_t *seq_lens;
} specv_kv_cache;

/* Append the keys and values of a pass to the cache, with rotary positions
 * applied on the way (the page's PagedKVCacheManager.append, and the depth
 * positions of "Multi-Draft Tree Speculation", s.3).  rows tokens a sequence:
 * row 0 follows the verified prefix, row 1 + i is draft node i.
 *   k, v        [B, rows, kv_heads, head_dim], element type cache->dtype;
 *               k_stride, v_stride elements from one row to the next (rows of
 *               a sequence and sequences alike), a multiple of 16 bytes
 *   q           as k, with q_heads heads (nullable: q_heads, q_stride and
 *               q_out are then not looked at)
 *   q_out       [B, rows, q_heads, head_dim] out, without gaps: q rotated; it
 *               may be q itself (q_stride = q_heads * head_dim).  Zero for
 *               padding rows, idle and refused sequences
 *   inv_freq    [rot_dim / 2] fp32: the first rot_dim (even, <= head_dim)
 *               values of each head of q and k turn in pairs by the angle
 *               position * inv_freq[j]; pair j is (j, j + rot_dim / 2), or
 *               (2j, 2j + 1) if interleaved.  rot_dim 0: no rotation
 *               (inv_freq may be NULL).  The angle is formed and brought into
 *               [-pi, pi] in float64; its sine and cosine and the products are
 *               fp32 (together off by at most 2^-21 of |x0| + |x1|), rounded
 *               once
 *   parents     [B, rows - 1] int32 as for specv_verify_tree_greedy; NULL:
 *               every sequence is a chain (then rows is not bounded by max_k,
 *               so that prompts can be appended)
 *   row_counts  [B] int32, 0..rows: the rows of each sequence that are tokens,
 *               the others being padding that is not read; NULL: all rows
 *               (none of an idle sequence).  Outside: bit 2048.  This is for
 *               prompts: specv_tree_attention and specv_cache_compact know no
 *               counts and take a sequence's last `rows` positions (last M)
 *               for the pass's, so that a pass whose counts are below rows is
 *               not one for them (they cannot tell; use a call for each count)
 *   row_status  [B] out (nullable): 0, or bits 512 (a parent outside
 *               [-1, i)), 2048, 4096.  Of a refused sequence nothing is written
 *               to the cache
 * Row r goes to cache position base + r, base = seq_lens - row count, and has
 * the rotary position base + depth(r): depth(0) = 0, a child one more than
 * its parent, so that a kept path keeps its rotation when specv_cache_compact
 * moves it.  Sequences of a batch must not share the blocks they write to, nor
 * a table name one of these twice. */
specv_status specv_cache_append(specv_handle h, const specv_kv_cache *cache, const void *q, int64_t q_stride,
                                int q_heads, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                const float *inv_freq, int rot_dim, int interleaved, const int32_t *parents,
                                const int32_t *row_counts, int batch, int rows, void *q_out, int32_t *row_status,
                                void *stream);

/* Attention of a pass's rows over the cache they were appended to ("LLM
 * Inference & Speculative Decoding: From Roofline Physics to Lossless
 * Acceleration", s.3, the ancestor mask): row r of a sequence sees every
 * position before the pass's rows, and of these itself and its ancestors
 * (row 0 is an ancestor of all).
 *   q           [B, rows, q_heads, head_dim], q_stride elements between rows;
 *               q_heads a multiple of kv_heads, query head h reads kv head
 *               h / (q_heads / kv_heads)
 *   parents     [B, rows - 1] int32; NULL: chains.  1 <= rows <= max_k + 1;
 *               rows = 1 is plain decoding
 *   scale       factor of the scores before the softmax; it and scale *
 *               log2(e), the factor of the scores in base 2, finite.  Scores
 *               are fp32: one that these take out of its range is infinite
 *   out         [B, rows, q_heads, head_dim] out, without gaps; not q's memory
 *   lse         [B, rows, q_heads] fp32 out (nullable): log of the sum of
 *               the exponentials of the scaled scores
 *   row_status  [B] out (nullable): 0, or bits 512, 2048, 4096, 64.  out of
 *               an idle or refused sequence is 0, lse -infinity; with bit 64
 *               what they hold of the sequence is not determined
 *   workspace   device memory of specv_tree_attention_workspace(...) bytes,
 *               256-byte aligned, the call's own until it has run
 * Positions that a row does not see take no part, whatever they hold (NaN and
 * infinities among them).  Sums are fp32.  Weights exp(score - m), with m at
 * most 8 log 2 below the row's largest score so far, are rounded to bf16 for the
 * product with the values of a bf16 cache (2^-9 each on average, 2^-8 at most,
 * so that an output is off by up to 2^-8 of the weighted mean of |v|, besides
 * its own rounding; their sum, and so lse, is not rounded); those of an fp32
 * cache, and its values, go in as two tf32 parts (products off by 3 * 2^-22 at
 * most).  Sums of weight * value are divided by the sum of the weights at the
 * end: of values above 2^119 or so they may leave fp32's range though the
 * result would not. */
specv_status specv_tree_attention(specv_handle h, const specv_kv_cache *cache, const void *q, int64_t q_stride,
                                  int q_heads, const int32_t *parents, int batch, int rows, float scale, void *out,
                                  float *lse, int32_t *row_status, void *workspace, int64_t workspace_bytes,
                                  void *stream);

/* Bytes of workspace that specv_tree_attention needs for these sizes (it does
 * not depend on lengths); 0 if none or if the sizes are invalid. */
int64_t specv_tree_attention_workspace(specv_handle h, specv_dtype dtype, int kv_heads, int head_dim, int q_heads,
                                       int batch, int rows);

/* specv_tree_attention for a batch whose sequences share a prefix (a system
 * prompt, a document): the prefix is read once for all of them.  Positions
 * before prefix_len are those of prefix_table, for every sequence; the others
 * are its own, by its block table (whose entries before prefix_len / block_size
 * are not looked at: they may name the same blocks, as the other calls need them).
 *   prefix_table  [prefix_blocks] int32
 *   prefix_len    [1] int32, device memory: positions of the prefix, a multiple
 *                 of block_size up to prefix_blocks * block_size; 0: none
 *   seq_lens      of the cache: whole lengths, the prefix's positions among them.
 *                 A sequence shorter than prefix_len + rows is refused
 *                 (bit 2048; 0 is idle as ever); so are all where prefix_len is
 *                 not as said (bit 2048) or an entry of prefix_table in use is
 *                 outside the pool (bit 4096)
 * Everything else, the roundings among it, as for specv_tree_attention;
 * workspace of specv_prefix_attention_workspace(...) bytes.  batch * rows *
 * q_heads * head_dim / 4 is below 2^31 - 128. */
specv_status specv_prefix_attention(specv_handle h, const specv_kv_cache *cache, const int32_t *prefix_table,
                                    int prefix_blocks, const int32_t *prefix_len, const void *q, int64_t q_stride,
                                    int q_heads, const int32_t *parents, int batch, int rows, float scale, void *out,
                                    float *lse, int32_t *row_status, void *workspace, int64_t workspace_bytes,
                                    void *stream);

/* Bytes of workspace that specv_prefix_attention needs for these sizes (it
 * does not depend on lengths); 0 if the sizes are invalid. */
int64_t specv_prefix_attention_workspace(specv_handle h, specv_dtype dtype, int kv_heads, int head_dim, int q_heads,
                                         int batch, int rows);

/* Move the kept path of a verified tree together in the cache, before
 * specv_rollback cuts the sequence off behind it: node path[i] (at position
 * seq_len - M + path[i]) is copied to position seq_len - M + i, for i <
 * num_accepted, in keys and values of `layers` layers at once (layer l of a
 * pool at l * layer_stride elements; 1 for a cache that is a tensor a layer).
 *   path, num_accepted  [B, M], [B] as specv_verify_tree_greedy gives them
 *   row_status          [B] out (nullable): 0, or bits 128 (num_accepted
 *                       outside [0, M]), 2048 (a length below M, 0 aside),
 *                       4096, 8192.  A refused sequence is left as it is
 * Positions behind the path keep what they held.  1 <= M <= max_k, layers >= 1. */
specv_status specv_cache_compact(specv_handle h, const specv_kv_cache *cache, int layers, int64_t layer_stride,
                                 const int32_t *path, const int32_t *num_accepted, int batch, int M,
                                 int32_t *row_status, void *stream);

/* Norms of the heads of an append (each weight nullable: those heads are
 * then not normed): a head x of queries or keys becomes x * rsqrt(mean(x^2) +
 * eps) * (weight + weight_add) before its pairs turn.  Weights [head_dim] of
 * the cache's type, device memory, 16-byte aligned; weight_add 1 for models that
 * keep weights as their difference from one, else 0.  eps >= 0 and weight_add
 * finite. */
typedef struct {
    const void *q_weight, *k_weight;
    float eps, weight_add;
} specv_head_norm;

/* Rotary positions of an append, where they are not base + depth.
 *   positions  [B, rows, axes] int32 (nullable): the position of each row on
 *              each axis (time, height and width of a patch of an image or
 *              video, say), any number.  Then offsets and parents are NULL
 *   axes       1..16
 *   pair_axis  [rot_dim / 2], HOST memory, read by the call: the axis, below
 *              axes, by whose position pair j turns (inv_freq[j] as ever).
 *              NULL with one axis
 *   offsets    [B] int32 (nullable; without positions): added to base + depth,
 *              for sequences whose positions run ahead of the cache (behind
 *              an eviction) or behind it (behind images) */
typedef struct {
    int axes;
    const int32_t *positions;
    const uint8_t *pair_axis;
    const int32_t *offsets;
} specv_positions;

/* specv_cache_append for models that norm the heads of queries and keys
 * and for positions on several axes: in addition `norm` and `positions`,
 * both nullable (and then exactly that call).  Norms, turns and products are fp32
 * with one rounding at the end; a head whose squares would leave fp32's range,
 * or vanish in it, is scaled by a power of two first, so that heads of any
 * finite values come out as the formula has them (one of zeros with eps 0 is
 * no number).  Everything else as there. */
specv_status specv_cache_append_norm(specv_handle h, const specv_kv_cache *cache, const void *q, int64_t q_stride,
                                     int q_heads, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                                     const specv_head_norm *norm, const float *inv_freq, int rot_dim, int interleaved,
                                     const specv_positions *positions, const int32_t *parents,
                                     const int32_t *row_counts, int batch, int rows, void *q_out, int32_t *row_status,
                                     void *stream);

/* The attention weight that the positions of a cache gather from a pass, for
 * specv_cache_evict: mass_out[b, h, t] = mass[b, h, t] + the sum, over the
 * pass's rows r that see position t and the query heads g of kv head h, of
 * exp(scale * q . k_t - lse[b, r, g]).
 *   q, q_stride, q_heads, parents, rows, scale  as for specv_tree_attention
 *   lse         [B, rows, q_heads] fp32, as specv_tree_attention (or
 *               specv_prefix_attention) left it.  A row whose lse is infinite
 *               takes no part
 *   path, num_accepted  [B, rows - 1], [B] (nullable) as a verify call gives
 *               them (path NULL: chains): rows of rejected drafts take no part,
 *               and a kept node's mass goes where specv_cache_compact moves its
 *               keys, behind this call; those behind the path are not written.
 *               Without num_accepted all rows stay
 *   mass        [B, kv_heads, width] fp32 (nullable: zeros).  The pass's own
 *               positions start from 0: what it holds there is not read
 *   mass_out    [B, kv_heads, width] fp32 out; mass itself, or memory apart
 *               from it.
 *               Written for positions first .. length - 1
 *   first       positions before it are left alone (a shared prefix).  Of a
 *               sequence that ends within the whole blocks before it only the
 *               length is looked at
 *   row_status  [B] out (nullable): 0, or bits 512, 2048 (also a length above
 *               width), 4096, 128 and 8192 (as for specv_cache_compact), 64.  Of
 *               a refused sequence nothing is written; with bit 64 what mass_out holds of it is not determined
 * Sums are fp32 in a fixed order: results repeat.  The values of the cache are
 * not read. */
specv_status specv_attention_mass(specv_handle h, const specv_kv_cache *cache, const void *q, int64_t q_stride,
                                  int q_heads, const int32_t *parents, int batch, int rows, float scale,
                                  const float *lse, const int32_t *path, const int32_t *num_accepted,
                                  const float *mass, float *mass_out, int64_t width, int first, int32_t *row_status,
                                  void *stream);

/* Eviction: sequences longer than `budget` are brought back to it, in keys and
 * values of `layers` layers at once (as specv_cache_compact counts them).  Of
 * each layer and kv head the first `first` and the last `recent` positions
 * stay, and of those between the budget - first - recent with the largest mass
 * (equal ones: the lower position; NaN counts as the largest).  Below line =
 * budget - recent kept positions stay where they are, the i-th hole there
 * takes the i-th kept position above, and the recent ones follow from the line
 * on in their order.  (Attention asks for no order among positions before a
 * pass; rotary positions are in the keys, and go on with specv_positions.offsets
 * raised by `evicted`.)
 *   mass        [layers, B, kv_heads, width] fp32 as specv_attention_mass
 *               gathers it
 *   mass_out    [layers, B, kv_heads, width] out: the masses of the positions
 *               that remain, at their places; memory apart from mass's.  Behind
 *               the new length it is left alone
 *   budget      1 or more, at least first + recent
 *   lens_out    [B] out: the new lengths.  It, evicted and row_status are memory
 *               apart from cache->seq_lens' and cache->block_tables'
 *   evicted     [B] out (nullable): old minus new length
 *   row_status  [B] out (nullable): 0, or bits 2048 (also a length above
 *               width or 2^31 - 4096), 4096 (an entry from position `first` on outside the
 *               pool).  Of a refused sequence nothing moves, and its length stays
 * Sequences must not share blocks from position `first` on.  Blocks that are
 * no longer in use stay in the tables: specv_rollback with these lengths and
 * num_accepted = k pops them into the free list. */
specv_status specv_cache_evict(specv_handle h, const specv_kv_cache *cache, int layers, int64_t layer_stride,
                               const float *mass, float *mass_out, int64_t width, int batch, int budget, int recent,
                               int first, int32_t *lens_out, int32_t *evicted, int32_t *row_status, void *stream);

/* Number of CTAs per sequence (thread-block cluster size, 1..16) that the
 * next call with these sizes would use; 0 if the sizes are invalid. */
int specv_plan_cluster(specv_handle h, specv_dtype logits_dtype, int batch, int k, int64_t V);

/* Test hook, off unless called: arms the next launch of the split-vocabulary
 * kernel (V > 2048), of the tcgen05 tree-attention kernel (bf16, head_dim up
 * to 128, more than 16 rows a kv head; of a shared prefix, more than 16 of the
 * batch: its own launch, or by numbers from 2^20 on, which then stand for 0 on,
 * the sequences') or of the tcgen05 kernel of specv_attention_mass (bf16,
 * head_dim up to 128, up to 256 rows a kv head) on this handle so that CTA 0 of the
 * grid never issues the bulk copy of its pass-1 stage use (the copies of its
 * slot use, or tile) number `stage_use` (counted from 0
 * in issue order) nor signals it, and every wait of that launch gives up
 * after `polls` polls.  The waits that run out end the row's work: it
 * reports row_status bit 64 (num_accepted 0, out_tokens -1) and the call
 * still returns SPECV_OK; the other rows and the next call run normally.  No
 * copy is in flight when a CTA exits (it waits, bounded, for every copy it
 * issued).  SPECV_ERR_INVALID_ARGUMENT for stage_use < 0 or polls < 1. */
specv_status specv_test_withhold_stage(specv_handle h, int stage_use, int polls);

/* Kernel launches issued by this handle since it was created. */
int64_t specv_launch_count(specv_handle h);

/* Release the handle and any buffers it owns.  NULL is ignored. */
void specv_destroy(specv_handle h);

/* Static description of a status code. */
const char *specv_status_string(specv_status s);

/* Text of the last CUDA error seen by this library on the calling thread. */
const char *specv_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SPECV_H */
