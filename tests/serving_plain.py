"""Plain float64 restatements of the calls for current models and long-running
batches on the paged KV cache, one sequence, row and head at a time: the
reference of the CUDA kernels.  The cache and the trees are those of
cache_plain.py."""
import numpy as np

import cache_plain as P
from cache_plain import ST_BLOCK, ST_LENGTH, ST_PARENT


def norm(x, weight, eps, add):
    """x [heads, dim] over the root of its mean square, times the weight."""
    x = np.asarray(x, np.float64)
    if weight is None:
        return x.copy()
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (np.asarray(weight, np.float64) + add)


def turn(x, angle, interleaved):
    """x [heads, dim] with its pairs turned by angle [pairs]."""
    x, half = np.array(x, np.float64), len(angle)
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        x0, x1 = x[:, i0].copy(), x[:, i1].copy()
        x[:, i0] = x0 * np.cos(angle[j]) - x1 * np.sin(angle[j])
        x[:, i1] = x0 * np.sin(angle[j]) + x1 * np.cos(angle[j])
    return x


def append_norm(kc, vc, tables, lens, k, v, *, q=None, q_norm=None, k_norm=None, eps=1e-6, add=0.0, inv_freq=None,
                interleaved=False, positions=None, axis=None, offsets=None, parents=None, counts=None):
    """kc, vc changed in place; returns (q_out, status, written, pairs): pairs
    has, for each written key and each query, |x0| + |x1| of the normed values
    that made each output, in arrays like kc and q."""
    B, rows = k.shape[:2]
    bs, cap = kc.shape[2], tables.shape[1] * kc.shape[2]
    q_out = None if q is None else np.zeros(q.shape)
    q_mag, k_mag = None if q is None else np.zeros(q.shape), np.zeros(kc.shape)
    status, written = np.zeros(B, np.int32), []
    freq = np.zeros(0) if inv_freq is None else np.asarray(inv_freq, np.float64)

    def mags(x):
        y, half = np.abs(x), len(freq)
        if half:
            a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
            both = y[:, a] + y[:, b]
            y[:, a] = y[:, b] = both
        return y

    for b in range(B):
        n = int(lens[b])
        m = int(counts[b]) if counts is not None else (0 if n == 0 else rows)
        if m < 0 or m > rows or n < 0 or (m > 0 and (n < m or n > cap)):
            status[b] = ST_LENGTH
            continue
        if m == 0:
            continue
        ok, depth, _ = P.tree(None if parents is None else parents[b], m)
        ids, inside = P.blocks_of(tables[b], n - m, n, bs, kc.shape[0])
        status[b] = (0 if ok else ST_PARENT) | (0 if inside else ST_BLOCK)
        if status[b]:
            continue
        for r in range(m):
            t = n - m + r
            if positions is not None:
                at = [int(positions[b, r, a]) for a in (axis if axis is not None else [0] * len(freq))]
            else:
                at = n - m + depth[r] + (0 if offsets is None else int(offsets[b]))
            angle = np.asarray(at, np.float64) * freq
            x = norm(k[b, r], k_norm, eps, add)
            kc[ids[r], :, t % bs], k_mag[ids[r], :, t % bs] = turn(x, angle, interleaved), mags(x)
            vc[ids[r], :, t % bs] = v[b, r]
            written.append((int(ids[r]), t % bs))
            if q is not None:
                x = norm(q[b, r], q_norm, eps, add)
                q_out[b, r], q_mag[b, r] = turn(x, angle, interleaved), mags(x)
    return q_out, status, written, (q_mag, k_mag)


def append_norm_bound(ref, mag, dim, half):
    """How far an output may be off.  The sum of dim squares adds at most dim
    roundings of 2^-24, its mean and eps two more; the root halves them; the
    reciprocal root is off by 2 units in the last place (2^-22), the weight,
    its product and the value's round once each (2^-24): the normed value is
    off by (dim / 2 + 1) 2^-24 + 2^-22 + 3 * 2^-24, relatively, of itself.  Its
    turn adds 2^-21 of |x0| + |x1| (as tests of the plain append derive), and
    the result is rounded once to its type (half of its step)."""
    e = (dim / 2 + 8) * 2.0 ** -24
    return half * np.abs(ref) + 1.01 * (e + 2.0 ** -21) * mag


def prefix_attention(q, kc, vc, tables, lens, prefix_table, prefix, parents, scale):
    """As cache_plain.attention over tables whose first blocks are the
    prefix's; (out, lse, status, avg, mag)."""
    bs, blocks = kc.shape[2], kc.shape[0]
    rows, B = q.shape[1], q.shape[0]
    lens = np.asarray(lens).copy()
    if prefix < 0 or prefix % bs or prefix > len(prefix_table) * bs:
        got = P.attention(q, kc, vc, tables, np.zeros_like(lens), parents, scale)
        got[2][lens != 0] = ST_LENGTH
        return got
    n = prefix // bs
    full = np.array(tables).copy()
    inside = np.all((prefix_table[:n] >= 0) & (prefix_table[:n] < blocks))
    refused = np.zeros(B, np.int32)
    for b in range(B):
        if lens[b] == 0:
            continue
        if lens[b] < prefix + rows or lens[b] > full.shape[1] * bs:
            refused[b] |= ST_LENGTH
        if not P.tree(None if parents is None else parents[b], rows)[0]:
            refused[b] |= ST_PARENT
        if not refused[b] & ST_LENGTH:  # (a bad tree and a bad block are both told)
            own = full[b, n:-(-int(lens[b]) // bs)]
            if not (inside and np.all((own >= 0) & (own < blocks))):
                refused[b] |= ST_BLOCK
        full[b, :n] = prefix_table[:n]
    out, lse, status, avg, mag = P.attention(q, kc, vc, full, np.where(refused, 0, lens), parents, scale)
    return out, lse, status | refused, avg, mag


def kept_of(path, accepted, rows):
    """(ok bits, rows that stay, their places) of one sequence's pass."""
    if accepted is None:
        return 0, list(range(rows)), list(range(rows))
    n = int(accepted)
    nodes = list(range(max(min(n, rows - 1), 0))) if path is None else [int(x) for x in path[:max(min(n, rows - 1), 0)]]
    bad = 0 if 0 <= n <= rows - 1 else P.ST_ACCEPTED
    if any(x < 0 or x >= rows - 1 for x in nodes) or any(y <= x for x, y in zip(nodes, nodes[1:])):
        bad |= P.ST_PATH
    return bad, [0] + [1 + x for x in nodes], list(range(len(nodes) + 1))


def mass(q, kc, tables, lens, lse, parents, scale, before, first, width, path=None, accepted=None):
    """Returns (gained [B, heads, width], status, written, bound): the new
    masses where written, and how far a kernel's may be off.

    A weight exp(s - lse): s is a sum of dim products in fp32 (2^-23 of the
    magnitudes a step; fp32 inputs enter as two tf32 parts, 3 * 2^-22 a
    product), times the scale; the exponent's argument, in base 2, rounds at
    the size of the score, of lse and of their product with log2 e (2^-23
    each); the exponential is off by 2^-21.  Sums of all weights add their
    number of roundings (2^-23 each, fp32)."""
    B, rows, hq, dim = q.shape
    heads, bs, cap = kc.shape[1], kc.shape[2], tables.shape[1] * kc.shape[2]
    group = hq // heads
    out, tol = np.zeros((B, heads, width)), np.zeros((B, heads, width))
    written, status = np.zeros((B, heads, width), bool), np.zeros(B, np.int32)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        if n < rows or n > cap or n > width:
            status[b] = ST_LENGTH
            continue
        skip = first // bs * bs
        if n <= skip:
            continue
        ok, _, seen = P.tree(None if parents is None else parents[b], rows)
        ids, inside = P.blocks_of(tables[b], skip, n, bs, kc.shape[0])
        bad, kept, places = kept_of(None if path is None else path[b], None if accepted is None else accepted[b], rows)
        status[b] = (0 if ok else ST_PARENT) | (0 if inside else ST_BLOCK) | bad
        if status[b]:
            continue
        K = kc[ids, :, np.arange(skip, n) % bs]  # [n - skip, heads, dim]
        for r in range(rows):
            see = np.array([t < n - rows or t - (n - rows) in seen[r] for t in range(skip, n)])
            for h in range(hq):
                l = float(lse[b, r, h])
                if np.isinf(l) or r not in kept:
                    continue
                kk = K[see, h // group]
                with np.errstate(all="ignore"):
                    s = kk @ q[b, r, h] * scale
                    w = np.exp(s - l)
                    size = np.abs(kk) @ np.abs(q[b, r, h]) * abs(scale)
                at = np.arange(skip, n)[see]
                out[b, h // group, at] += w
                tol[b, h // group, at] += w * ((dim + 16) * 2.0 ** -23 * size + 2.0 ** -22 * (np.abs(s) + 2 * abs(l))
                                               + 2.0 ** -21)
        tol[b] += out[b] * (rows * group + 8) * 2.0 ** -23
        if before is not None:
            out[b, :, :n - rows] += before[b, :, :n - rows]
            tol[b, :, :n - rows] += np.abs(out[b, :, :n - rows]) * 2.0 ** -23
        written[b, :, first:n] = True
        if accepted is not None:  # kept nodes to their places, the others nowhere
            base = n - rows
            for x in (out, tol):
                x[b, :, base:base + len(kept)] = x[b, :, [base + r for r in kept]].T
            written[b, :, base:n] = False
            for r, to in zip(kept, places):
                written[b, :, base + to] = base + to >= first
    return out, status, written, 1.01 * tol


def evict(kc, vc, tables, lens, mass, budget, recent, first):
    """kc, vc [layers, blocks, heads, bs, dim], changed in place, mass [layers,
    B, heads, width]; returns (places, new lens, status): places [layers][B][heads] the old
    position of each position that remains (None: all stay)."""
    layers, B, heads, width = mass.shape
    bs, cap = kc.shape[3], tables.shape[1] * kc.shape[3]
    new, status = np.array(lens).copy(), np.zeros(B, np.int32)
    places = [[[None] * heads for _ in range(B)] for _ in range(layers)]
    line = budget - recent
    for b in range(B):
        n = int(lens[b])
        if n < 0 or n > cap or n > width:
            status[b] = ST_LENGTH
            continue
        if n <= budget:
            continue
        if not P.blocks_of(tables[b], first // bs * bs, n, bs, kc.shape[1])[1]:
            status[b] = ST_BLOCK
            continue
        new[b] = budget
        for l in range(layers):
            for h in range(heads):
                row = [float(x) for x in mass[l, b, h, :n]]
                open_ = range(first, n - recent)
                worth = [np.inf if np.isnan(x) else x for x in row]
                nan = [np.isnan(x) for x in row]
                kept = set(sorted(open_, key=lambda t: (not nan[t], -worth[t], t))[:line - first])
                holes = [t for t in range(first, line) if t not in kept]
                above = [t for t in range(line, n - recent) if t in kept]
                assert len(holes) == len(above)
                place = list(range(line)) + list(range(n - recent, n))
                for t, s in zip(holes, above):
                    place[t] = s
                places[l][b][h] = place
                t, s = np.arange(budget), np.array(place)
                for c in (kc, vc):
                    c[l, tables[b, t // bs], h, t % bs] = c[l, tables[b, s // bs], h, s % bs]
    return places, new, status
