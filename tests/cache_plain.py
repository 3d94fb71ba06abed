"""Plain float64 restatements of the calls on the paged KV cache, one
sequence, row and head at a time: the checker of the CUDA kernels.

"LLM Inference & Speculative Decoding: From Roofline Physics to Lossless
Acceleration", s.1 (PagedKVCacheManager: position t is in block t /
block_size of the sequence's table, at t % block_size) and s.3 (ancestor mask
and depths from a parent array)."""
import numpy as np

ST_ACCEPTED, ST_PARENT, ST_LENGTH, ST_BLOCK, ST_PATH = 128, 512, 2048, 4096, 8192


def tree(parents, rows):
    """(ok, depth [rows], seen [rows][..]) of one sequence's rows; parents
    None: a chain.  seen[r] lists row r and the rows above it."""
    depth, seen, ok = [0], [[0]], True
    for i in range(rows - 1):
        p = i - 1 if parents is None else int(parents[i])
        if not -1 <= p < i:
            ok = False
            p = -1
        depth.append(depth[p + 1] + 1)
        seen.append(seen[p + 1] + [i + 1])
    return ok, depth, seen


def blocks_of(table, lo, hi, bs, blocks):
    """Physical block of positions lo..hi-1, and whether all are in the pool."""
    ids = np.array([int(table[t // bs]) for t in range(lo, hi)], np.int64)
    return ids, bool(np.all((ids >= 0) & (ids < blocks)))


def rotate(x, pos, inv_freq, interleaved):
    """x [heads, dim] float64 turned by pos."""
    x = np.array(x, np.float64)
    half = 0 if inv_freq is None else len(inv_freq)
    for j in range(half):
        a = float(pos) * float(inv_freq[j])
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        x0, x1 = x[:, i0].copy(), x[:, i1].copy()
        x[:, i0] = x0 * np.cos(a) - x1 * np.sin(a)
        x[:, i1] = x0 * np.sin(a) + x1 * np.cos(a)
    return x


def append(kc, vc, tables, lens, k, v, *, q=None, inv_freq=None, interleaved=False, parents=None, counts=None):
    """kc, vc [blocks, heads, bs, dim] float64, changed in place; returns
    (q_out, status, written) with written a list of (block, slot)."""
    B, rows = k.shape[:2]
    bs, cap = kc.shape[2], tables.shape[1] * kc.shape[2]
    q_out = None if q is None else np.zeros(q.shape)
    status, written = np.zeros(B, np.int32), []
    for b in range(B):
        n = int(lens[b])
        m = int(counts[b]) if counts is not None else (0 if n == 0 else rows)
        if m < 0 or m > rows or n < 0 or (m > 0 and (n < m or n > cap)):
            status[b] = ST_LENGTH
            continue
        if m == 0:
            continue
        ok, depth, _ = tree(None if parents is None else parents[b], m)
        ids, inside = blocks_of(tables[b], n - m, n, bs, kc.shape[0])
        status[b] = (0 if ok else ST_PARENT) | (0 if inside else ST_BLOCK)
        if status[b]:
            continue
        for r in range(m):
            t = n - m + r
            kc[ids[r], :, t % bs] = rotate(k[b, r], n - m + depth[r], inv_freq, interleaved)
            vc[ids[r], :, t % bs] = v[b, r]
            written.append((int(ids[r]), t % bs))
            if q is not None:
                q_out[b, r] = rotate(q[b, r], n - m + depth[r], inv_freq, interleaved)
    return q_out, status, written


def attention(q, kc, vc, tables, lens, parents, scale):
    """Returns out, lse, status and two bounds' ingredients: avg [like out],
    the mean of |v| under the same weights, and mag [B, rows, heads], the
    largest sum |q_d k_d| * |scale| of a row."""
    B, rows, hq, dim = q.shape
    bs, heads, cap = kc.shape[2], kc.shape[1], tables.shape[1] * kc.shape[2]
    out, avg = np.zeros(q.shape), np.zeros(q.shape)
    lse, mag = np.full((B, rows, hq), -np.inf), np.zeros((B, rows, hq))
    status = np.zeros(B, np.int32)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        if n < rows or n > cap:
            status[b] = ST_LENGTH
        ok, _, seen = tree(None if parents is None else parents[b], rows)
        if not ok:
            status[b] |= ST_PARENT
        if status[b]:
            continue
        ids, inside = blocks_of(tables[b], 0, n, bs, kc.shape[0])
        if not inside:
            status[b] = ST_BLOCK
            continue
        K, V = kc[ids, :, np.arange(n) % bs], vc[ids, :, np.arange(n) % bs]  # [n, heads, dim]
        for r in range(rows):
            at = list(range(n - rows)) + [n - rows + j for j in sorted(seen[r])]
            for h in range(hq):
                kk, vv = K[at, h // (hq // heads)], V[at, h // (hq // heads)]
                with np.errstate(all="ignore"):
                    s = kk @ q[b, r, h] * scale
                    m = np.max(s)
                    p = np.exp(s - m)
                    out[b, r, h] = (p @ vv) / p.sum()
                    avg[b, r, h] = (p @ np.abs(vv)) / p.sum()
                    lse[b, r, h] = m + np.log(p.sum())
                    mag[b, r, h] = np.max(np.abs(kk) @ np.abs(q[b, r, h])) * abs(scale)
    return out, lse, status, avg, mag


def attention_bounds(out, lse, avg, mag, n_max, dim, bf16):
    """How far a kernel's outputs may be off, from its arithmetic:

    a score is a sum of dim products in fp32 (each step off by at most 2^-23
    of the magnitudes, truncation included; fp32 inputs enter the tensor cores
    as two tf32 parts, off by 3 * 2^-22 of the product), times the scale (one
    rounding): e_s = (dim + 16) * 2^-23 * mag.  The exponential's argument is
    rounded at the size of the scores (2 * mag * 2^-23), the exponential
    itself is off by 2^-21: p is off by e = e_s + mag * 2^-22 + 2^-21,
    relatively.  Weights of bf16 values are rounded to bf16 (2^-8).  Sums over
    the n positions, and over rescaled parts of them, add (n + 64) * 2^-23 at
    most.  o is a mean of v under p: numerator and denominator are each off by
    these, and the result is rounded once to its type."""
    eps = 2.0 ** -8 if bf16 else 2.0 ** -24
    e = (dim + 16) * 2.0 ** -23 * mag + mag * 2.0 ** -22 + 2.0 ** -21
    n = (n_max + 64) * 2.0 ** -23
    weight = 2.0 ** -8 if bf16 else 3 * 2.0 ** -22
    tol = eps * np.abs(out) + (1.01 * (2 * e + 2 * n + weight))[..., None] * avg
    return tol, e + n + 2.0 ** -23 * np.abs(lse) + 2.0 ** -22


def compact(kc, vc, tables, lens, path, num_accepted):
    """kc, vc [layers, blocks, heads, bs, dim], changed in place; status."""
    B, M = path.shape
    bs, cap = kc.shape[3], tables.shape[1] * kc.shape[3]
    status = np.zeros(B, np.int32)
    for b in range(B):
        n, a = int(lens[b]), int(num_accepted[b])
        if n == 0:
            continue
        if a < 0 or a > M:
            status[b] |= ST_ACCEPTED
        if n < M or n > cap:
            status[b] |= ST_LENGTH
        if status[b]:
            continue
        p = [int(x) for x in path[b, :a]]
        if any(x < 0 or x >= M for x in p) or any(y <= x for x, y in zip(p, p[1:])):
            status[b] = ST_PATH
            continue
        moves = [(n - M + x, n - M + i) for i, x in enumerate(p)]
        used = [int(tables[b][t // bs]) for m in moves for t in m]
        if any(x < 0 or x >= kc.shape[1] for x in used):
            status[b] = ST_BLOCK
            continue
        for src, dst in moves:
            for c in (kc, vc):
                c[:, tables[b][dst // bs], :, dst % bs] = c[:, tables[b][src // bs], :, src % bs]
    return status
