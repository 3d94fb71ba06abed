"""Cases for more operators on the paged KV cache: append with a norm of every head and
positions on several axes, attention over a prefix that the batch shares, the attention
weight that positions gather, eviction by it.

A cache is a pool of blocks [blocks, kv_heads, block_size, head_dim] for keys and one
for values; row b of the block table names the blocks of sequence b, and seq_lens[b] is
the number of positions it holds, the rows of the current pass the last of them.  Row 0
of a pass is the token after the verified prefix, row 1 + i is draft node i; parents[i]
is a node, or -1 for a child of row 0.
"""
import functools
import math

import torch

own = False


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step without drafts of a model that norms its queries and keys
        dict(name="norm token", op="append", dtype="bf16", batch=8, rows=1, tree=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, rot=128, interleaved=False, axes=0, norm=True, offset=False, length=2000,
             ragged=False),
        # a draft tree for every sequence of a serving batch whose caches were shortened before: positions run ahead
        dict(name="norm tree", op="append", dtype="bf16", batch=64, rows=17, tree=True, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, rot=128, interleaved=False, axes=0, norm=True, offset=True, length=1000,
             ragged=False),
        # ragged prompts with images: time, height and width have pairs of their own
        dict(name="norm image prompt", op="append", dtype="bf16", batch=4, rows=2048, tree=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, rot=128, interleaved=False, axes=3, norm=True, offset=False, length=2500,
             ragged=True),
        # a small fp32 draft model: chains of 4, half of the head rotated, interleaved pairs
        dict(name="norm f32", op="append", dtype="f32", batch=16, rows=5, tree=False, q_heads=12, kv_heads=12,
             head_dim=64, block_size=16, rot=32, interleaved=True, axes=0, norm=True, offset=False, length=700,
             ragged=False),
        # one new token for each sequence of a batch behind one system prompt
        dict(name="prefix token", op="prefix", dtype="bf16", batch=64, rows=1, tree=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, prefix=4096, length=500, lse=False),
        # draft trees in the same batch, a longer prompt
        dict(name="prefix tree", op="prefix", dtype="bf16", batch=64, rows=17, tree=True, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, prefix=8192, length=1000, lse=True),
        # a few questions to one long document
        dict(name="prefix document", op="prefix", dtype="bf16", batch=16, rows=6, tree=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, prefix=65536, length=500, lse=False),
        # the fp32 draft model behind a short system prompt
        dict(name="prefix f32", op="prefix", dtype="f32", batch=8, rows=5, tree=False, q_heads=12, kv_heads=12,
             head_dim=64, block_size=16, prefix=1024, length=300, lse=False),
        # what the positions of a batch gather in a decode step
        dict(name="mass token", op="mass", dtype="bf16", batch=64, rows=1, tree=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, length=2000, first=0, start=False),
        # ... and in a pass of draft trees over longer contexts, a system prompt left alone
        dict(name="mass tree", op="mass", dtype="bf16", batch=64, rows=17, tree=True, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, length=4096, first=64, start=False),
        # one layer of a small batch is brought back to its budget
        dict(name="evict layer", op="evict", dtype="bf16", batch=8, layers=1, kv_heads=8, head_dim=128, block_size=16,
             length=1500, budget=1024, recent=256, first=4),
        # a batch of longer contexts, many layers at once
        dict(name="evict layers", op="evict", dtype="bf16", batch=32, layers=8, kv_heads=8, head_dim=128, block_size=16,
             length=2048, budget=1024, recent=256, first=4),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "prefix", "prefix", "mass", "evict"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    c = dict(op=op, dtype=dtype, batch=_spread(rng, 1, 128), kv_heads=rng.choice([1, 2, 4, 8, 10]),
             head_dim=rng.choice([64, 64, 96, 128, 128, 128, 256]), block_size=rng.choice([5, 8, 16, 16, 16, 32, 64]))
    line = c["kv_heads"] * c["head_dim"] * size  # bytes of one position of one cache
    if op == "evict":
        c["first"], c["recent"] = rng.choice([0, 0, 4, 64]), _spread(rng, 1, 400)
        c["budget"] = c["first"] + c["recent"] + _spread(rng, 1, 1500)
        c["length"] = c["budget"] + c["recent"] + _spread(rng, 1, 2000)
        c["batch"] = max(1, min(c["batch"], int(6e8 / (c["length"] * line))))
        c["layers"] = _spread(rng, 1, max(1, min(32, int(6e8 / (c["batch"] * (c["length"] + 64) * line)))))
        return c
    c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 4, 5, 8])
    c["tree"] = rng.random() < 0.6
    if op == "append":
        c["rows"] = rng.randint(1, 32) if c["tree"] else _spread(rng, 1, 2048)
        tokens = int(1.2e8 / (line * (1 + c["q_heads"] // c["kv_heads"])))
        c["batch"] = max(1, min(c["batch"], tokens // c["rows"], int(2.5e8 / (1200 * line))))
        c["rows"] = min(c["rows"], tokens)
        c["rot"] = rng.choice([c["head_dim"], c["head_dim"], c["head_dim"] // 2])
        c["interleaved"] = rng.random() < 0.3
        c["norm"] = rng.random() < 0.8
        c["axes"] = rng.choice([1, 2, 3, 3]) if not c["tree"] and rng.random() < 0.7 else 0
        c["offset"] = not c["axes"] and rng.random() < 0.5
        c["ragged"] = not c["tree"] and rng.random() < 0.7
        c["length"] = c["rows"] + _spread(rng, 1, 1000)
        return c
    c["rows"] = rng.randint(1, 32)
    if op == "mass":
        # no more bytes, and no more products, than the largest listed case
        keys = min(8e8 / line, 4e11 / (2 * c["rows"] * c["q_heads"] * c["head_dim"]))
        if dtype == "f32":
            keys /= 8
        c["length"] = _spread(rng, c["rows"], max(c["rows"], min(65536, int(keys))))
        c["batch"] = max(1, min(c["batch"], int(keys / c["length"])))
        c["first"] = rng.choice([0, 0, 4, 64])
        c["start"] = rng.random() < 0.3
        return c
    products = 1.4e11 / (4 * c["rows"] * c["q_heads"] * c["head_dim"])  # pairs of a sequence and a position
    if dtype == "f32":
        products /= 16
    c["length"] = _spread(rng, c["rows"], max(c["rows"], min(2000, int(products / 4))))
    c["batch"] = max(1, min(c["batch"], int(products / (4 * c["length"]))))
    blocks = _spread(rng, 1, max(1, min(65536, int(products * 0.7 / c["batch"])) // c["block_size"]))
    c["prefix"] = blocks * c["block_size"]
    c["lse"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------- inputs
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pool(shape, dtype, g):
    """A pool of keys or values, leftovers of earlier sequences in the positions that none holds."""
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def _tables(lens, block_size, g, shared=0):
    """Blocks for sequences of these lengths, shuffled over a pool with some to spare, -1 behind the last; the first
    `shared` blocks are the same in all."""
    used = [(n + block_size - 1) // block_size for n in lens]
    total = shared + len(lens) * (max(used) - shared) + 7
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32)
    table[:, :shared] = order[:shared]
    at = shared
    for b, n in enumerate(used):
        table[b, shared:n] = order[at:at + n - shared]
        at += n - shared
    return table.cuda(), total


def _lengths(case, least, g):
    """The first sequence at the full length, the others from half of it up."""
    n = torch.randint(max(least, case["length"] // 2), max(least, case["length"]) + 1, (case["batch"],), generator=g)
    n[0] = max(least, case["length"])
    return n


def _random_parents(batch, nodes, g):
    """parents[b, i] anywhere in -1..i-1."""
    pick = torch.rand((batch, nodes), generator=g, dtype=torch.float64)
    return torch.floor(pick * (torch.arange(nodes) + 1)).to(torch.int32) - 1


def _image_positions(batch, rows, axes, g):
    """[B, rows, axes]: text, an image of a few dozen patches a side, text again, which goes on behind the largest."""
    text = torch.randint(0, rows // 3 + 1, (batch, 1), generator=g)
    wide = torch.randint(8, 41, (batch, 1), generator=g)
    at = torch.arange(rows)[None] - text
    high = (rows // 2) // wide + 1
    inside = (at >= 0) & (at < high * wide)
    axis = [torch.zeros_like(at), at // wide, at % wide]
    behind = at - high * wide + torch.maximum(high, wide)
    place = [torch.where(inside, x, torch.where(at < 0, at, behind)) + text for x in axis]
    return torch.stack(place[3 - axes:], -1).to(torch.int32).contiguous()


def _pair_axis(pairs, axes):
    """A quarter of the pairs turns by the first of three axes, the rest is shared; fewer axes: even shares."""
    if axes == 3:
        first = pairs // 4
        return [0] * first + [1] * ((pairs - first) // 2) + [2] * (pairs - first - (pairs - first) // 2)
    return [j * axes // pairs for j in range(pairs)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.Generator().manual_seed(seed)
    dtype, batch = _type(case), case["batch"]
    heads, dim, bs = case["kv_heads"], case["head_dim"], case["block_size"]
    s = dict(case=case, status=torch.empty(batch, dtype=torch.int32, device="cuda"))
    if case["op"] == "evict":
        # no place that is written is read too, so that a pass can be repeated on the same caches: a sequence that is over
        # its budget is so by `recent` positions at least, and those that lie where the recent ones go, late ones, have
        # gathered little
        budget, recent, first, layers = case["budget"], case["recent"], case["first"], case["layers"]
        lens = torch.randint(budget + recent, case["length"] + 1, (batch,), generator=c)
        lens = torch.where(torch.rand(batch, generator=c) < 0.1, torch.randint(1, budget + 1, (batch,), generator=c), lens)
        lens[0] = case["length"]
        s["tables"], total = _tables(lens.tolist(), bs, c)
        s["lens"] = lens.to(torch.int32).cuda()
        s["k_cache"] = _pool((layers, total, heads, bs, dim), dtype, g)
        s["v_cache"] = _pool((layers, total, heads, bs, dim), dtype, g)
        width = s["tables"].shape[1] * bs
        # few positions gather most of the weight
        mass = torch.empty((layers, batch, heads, width), device="cuda").exponential_(generator=g) ** 3
        mass[..., budget - recent:budget] = 0.0
        s["mass"] = mass
        s["out"] = dict(mass=torch.zeros_like(mass), seq_lens=torch.zeros_like(s["lens"]),
                        evicted=torch.zeros_like(s["lens"]), row_status=s["status"])
        return s
    rows, q_heads = case["rows"], case["q_heads"]
    s["parents"] = _random_parents(batch, rows - 1, c).cuda() if case["tree"] else None
    prefix = case["prefix"] if case["op"] == "prefix" else 0
    lens = _lengths(case, rows, c) + prefix
    if case["op"] == "append":
        s["counts"] = None
        if case["ragged"]:
            counts = torch.randint(1, rows + 1, (batch,), generator=c)
            counts[0] = rows
            lens = lens - rows + counts
            s["counts"] = counts.to(torch.int32).cuda()
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        s["positions"] = s["axis"] = s["offsets"] = None
        if case["axes"]:
            s["positions"] = _image_positions(batch, rows, case["axes"], c).cuda()
            s["axis"] = bytes(_pair_axis(half, case["axes"]))
        if case["offset"]:
            s["offsets"] = torch.randint(0, 5000, (batch,), generator=c, dtype=torch.int32).cuda()
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"], s["k_norm"] = (torch.rand(dim, generator=g, device="cuda").add(0.5).to(dtype) for _ in range(2))
    s["tables"], total = _tables(lens.tolist(), bs, c, prefix // bs)
    s["lens"] = lens.to(torch.int32).cuda()
    s["k_cache"] = _pool((total, heads, bs, dim), dtype, g)
    s["v_cache"] = _pool((total, heads, bs, dim), dtype, g)
    # queries, keys and values lie behind one another, as one product of the hidden state gives them
    fused = torch.randn((batch, rows, q_heads + 2 * heads, dim), generator=g, device="cuda")
    fused[:, :, :q_heads] *= 2  # scores that spread by two: a few positions of a context carry most of the weight
    fused = fused.to(dtype)
    s["q"], s["k"], s["v"] = fused[:, :, :q_heads], fused[:, :, q_heads:q_heads + heads], fused[:, :, q_heads + heads:]
    s["out"] = {"row_status": s["status"]}
    if case["op"] == "mass":
        width = s["tables"].shape[1] * bs
        s["mass"] = None if case["start"] else torch.rand((batch, heads, width), generator=g, device="cuda")
        s["out"]["mass"] = torch.zeros((batch, heads, width), device="cuda")
        s["lse"] = _sums(s)  # as the attention over the same cache leaves it
        return s
    name = "q_out" if case["op"] == "append" else "out"
    s["out"][name] = torch.empty((batch, rows, q_heads, dim), dtype=dtype, device="cuda")
    if case["op"] == "prefix":
        s["prefix_table"] = s["tables"][0, :prefix // bs].clone()
        s["prefix_len"] = torch.tensor([prefix], dtype=torch.int32, device="cuda")
        if case["lse"]:
            s["out"]["lse"] = torch.empty((batch, rows, q_heads), dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms
def _reach(parents, batch, rows):
    """[B, R, R]: whether column j is row i or above it in the tree; None stands for chains."""
    at = torch.arange(rows, device="cuda")
    if parents is None:
        return (at[None, :] <= at[:, None]).expand(batch, rows, rows)
    up = torch.zeros((batch, rows, rows), device="cuda")
    up[:, 1:].scatter_(2, (parents.long() + 1)[:, :, None], 1.0)
    up = up + torch.eye(rows, device="cuda")
    up = up @ up
    up = up @ up
    up = up @ up
    up = up @ up
    up = up @ up  # paths of up to 32 steps
    return up > 0


def _normed(x, weight, eps=1e-6):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()


def _rotate(x, angle, interleaved):
    """x [B, R, H, D] rotated in its first pairs by angle [B, R, pairs], in 64 bits."""
    half = angle.shape[-1]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    x, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    a, b = a * cos - b * sin, a * sin + b * cos
    x = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((x, rest), -1)


def _plain_append(s):
    case, dtype, bs = s["case"], s["k_cache"].dtype, s["case"]["block_size"]
    batch, rows = case["batch"], case["rows"]
    at = torch.arange(rows, device="cuda")
    counts = torch.full_like(s["lens"], rows) if s["counts"] is None else s["counts"]
    base = (s["lens"] - counts).long()
    if s["positions"] is not None:
        pos = s["positions"].double()[:, :, list(s["axis"])]
    else:
        depth = at.expand(batch, rows) if s["parents"] is None else _reach(s["parents"], batch, rows).sum(-1) - 1
        pos = (base[:, None] + depth).double()[:, :, None]
        if s["offsets"] is not None:
            pos = pos + s["offsets"][:, None, None]
    angle = pos * s["inv_freq"].double()
    real = at < counts[:, None]
    q = _rotate(_normed(s["q"], s["q_norm"]), angle, case["interleaved"]).to(dtype)
    q = torch.where(real[:, :, None, None], q, torch.zeros((), dtype=dtype, device="cuda"))
    k = _rotate(_normed(s["k"], s["k_norm"]), angle, case["interleaved"]).to(dtype)
    # rows behind a sequence's last write what its row 0 writes, once more
    row = torch.where(real, at, 0)
    slot = base[:, None] + row
    block = s["tables"].long().gather(1, slot // bs)
    pick = row[:, :, None, None]
    s["k_cache"][block, :, slot % bs] = torch.take_along_dim(k, pick, 1)
    s["v_cache"][block, :, slot % bs] = torch.take_along_dim(s["v"], pick, 1)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _lines(cache, table):
    """[.., heads, positions, dim] in 32 bits, of the blocks of a table."""
    x = cache[table.long().clamp(min=0)]
    return x.transpose(-4, -3).flatten(-3, -2).float()


def _by_head(s):
    """Queries [B, kv_heads, rows * group, dim] in 32 bits."""
    case = s["case"]
    batch, rows, heads, dim = case["batch"], case["rows"], case["kv_heads"], case["head_dim"]
    q = s["q"].float().reshape(batch, rows, heads, -1, dim)
    return q.permute(0, 2, 1, 3, 4).reshape(batch, heads, -1, dim)


def _own_scores(s, k, skip):
    """Scores [B, heads, rows, group, positions] of the positions from `skip` on, -inf where a row does not see one."""
    case, rows = s["case"], s["case"]["rows"]
    n = k.shape[2]
    node = torch.arange(skip, skip + n, device="cuda") - (s["lens"].long() - rows)[:, None]
    seen = _reach(s["parents"], case["batch"], rows).gather(
        2, node.clamp(0, rows - 1)[:, None].expand(case["batch"], rows, n))
    seen = (node < 0)[:, None] | (seen & (node < rows)[:, None])
    x = (_by_head(s) @ k.transpose(2, 3)).mul_(1 / math.sqrt(case["head_dim"]))
    x = x.view(case["batch"], case["kv_heads"], rows, -1, n)
    return x.masked_fill_(~seen[:, None, :, None], -math.inf)


def _back(x, case):
    """[B, heads, rows, group, ..] as [B, rows, q_heads, ..]."""
    return x.transpose(1, 2).flatten(2, 3)


def _plain_prefix(s):
    case, bs = s["case"], s["case"]["block_size"]
    batch, rows, heads, dim = case["batch"], case["rows"], case["kv_heads"], case["head_dim"]
    skip = case["prefix"]
    k0, v0 = _lines(s["k_cache"], s["prefix_table"]), _lines(s["v_cache"], s["prefix_table"])  # [heads, prefix, dim]
    table = s["tables"][:, skip // bs:]
    k, v = _lines(s["k_cache"], table), _lines(s["v_cache"], table)
    x = _own_scores(s, k, skip)
    q0 = _by_head(s).transpose(0, 1).reshape(heads, -1, dim)
    x0 = (q0 @ k0.transpose(1, 2)).mul_(1 / math.sqrt(dim))
    shape = (heads, batch, rows, -1)
    top0 = x0.amax(-1).view(shape).transpose(0, 1)
    top = torch.maximum(x.amax(-1), top0)
    x0.sub_(top.transpose(0, 1).reshape(heads, -1, 1)).exp_()
    x.sub_(top[..., None]).exp_()
    total = x.sum(-1) + x0.sum(-1).view(shape).transpose(0, 1)
    o = (x.flatten(2, 3) @ v).view(batch, heads, rows, -1, dim)
    o += (x0 @ v0).view(heads, batch, rows, -1, dim).transpose(0, 1)
    got = {"out": _back(o / total[..., None], case).to(s["q"].dtype)}
    if case["lse"]:
        got["lse"] = _back(top + total.log(), case).contiguous()
    return got


def _sums(s):
    """Log of the sum of the exponentials of a row's scores, [B, rows, q_heads]."""
    x = _own_scores(s, _lines(s["k_cache"], s["tables"]), 0)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    return _back(top[..., 0] + x.sum(-1).log(), s["case"]).contiguous()


def _plain_mass(s):
    case, rows, heads = s["case"], s["case"]["rows"], s["case"]["kv_heads"]
    x = _own_scores(s, _lines(s["k_cache"], s["tables"]), 0)
    lse = s["lse"].view(case["batch"], rows, heads, -1).transpose(1, 2)
    gained = x.sub_(lse[..., None]).exp_().sum((2, 3))  # [B, heads, positions]
    at = torch.arange(gained.shape[2], device="cuda")[None]
    lens = s["lens"][:, None]
    if s["mass"] is not None:
        gained = gained + torch.where((at < lens - rows)[:, None], s["mass"], 0.0)
    written = ((at >= case["first"]) & (at < lens))[:, None]
    out = s["out"]["mass"]
    out.copy_(torch.where(written, gained, out))
    return {"mass": out}


def _plain_evict(s):
    case, bs = s["case"], s["case"]["block_size"]
    budget, recent, first = case["budget"], case["recent"], case["first"]
    line = budget - recent  # where the recent ones go to
    mass, lens = s["mass"], s["lens"].long()
    width = mass.shape[-1]
    at = torch.arange(width, device="cuda")
    over = lens > budget
    tail = (lens - recent)[:, None]
    open_ = ((at >= first) & (at < tail))[None, :, None]  # [1, B, 1, positions]
    # the largest first, the lowest position first among equals
    order = torch.where(open_, mass, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(mass, dtype=torch.bool)
    kept.scatter_(-1, order[..., :line - first], True)
    kept &= open_
    # holes below the line, in order, take the kept ones above it, in order; what has no place to go to stays
    big = torch.full_like(order, width)
    holes = torch.where(~kept & (at >= first) & (at < line), at, big).sort(-1).values[..., :line - first]
    above = torch.where(kept & (at >= line), at, big).sort(-1).values[..., :line - first]
    moving = (above < width) & over[:, None, None]
    last = torch.arange(recent, device="cuda").expand(*mass.shape[:3], recent)
    src = torch.cat((torch.where(moving, above, 0), torch.where(over[:, None, None], tail[:, :, None], line) + last), -1)
    dst = torch.cat((torch.where(moving, holes, 0), line + last), -1)
    go = torch.cat((moving, over[:, None, None].expand_as(last)), -1)
    src = torch.where(go, src, 0)
    dst = torch.where(go, dst, 0)
    real = go.nonzero(as_tuple=True)
    src, dst = src[real], dst[real]
    layer, seq, head, _ = real
    table = s["tables"].long()
    a, b = table[seq, src // bs], table[seq, dst // bs]
    s["k_cache"][layer, b, head, dst % bs] = s["k_cache"][layer, a, head, src % bs]
    s["v_cache"][layer, b, head, dst % bs] = s["v_cache"][layer, a, head, src % bs]
    out = s["out"]
    ends = torch.where(over, budget, lens)
    out["mass"].copy_(torch.where((at < ends[:, None])[None, :, None], mass, out["mass"]))
    out["mass"][layer, seq, head, dst] = mass[layer, seq, head, src]
    out["seq_lens"].copy_(ends)
    out["evicted"].copy_(lens - ends)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "mass": out["mass"], "seq_lens": out["seq_lens"],
            "evicted": out["evicted"]}


# ---------------------------------------------------------------------------- the framework's calls
@functools.lru_cache(maxsize=None)
def _handle():
    import speculative_decoding_verification_57_gb300 as sv

    return sv, sv.specv_create(0, max_batch=256, max_k=31)


def _own_append(s):
    sv, h = _handle()
    out = sv.specv_cache_append_norm(h, s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["k"], s["v"], q=s["q"],
                                     q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6, inv_freq=s["inv_freq"],
                                     interleaved=s["case"]["interleaved"], positions=s["positions"],
                                     pair_axis=s["axis"], offsets=s["offsets"], parents=s["parents"],
                                     row_counts=s["counts"], out=s["out"])
    return {"q": out["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_prefix(s):
    sv, h = _handle()
    out = sv.specv_prefix_attention(h, s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["prefix_table"],
                                    s["prefix_len"], parents=s["parents"], lse=s["case"]["lse"], out=s["out"])
    return {"out": out["out"], "lse": out["lse"]} if s["case"]["lse"] else {"out": out["out"]}


def _own_mass(s):
    sv, h = _handle()
    out = sv.specv_attention_mass(h, s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["lse"],
                                  mass=s["mass"], first=s["case"]["first"], parents=s["parents"], out=s["out"])
    return {"mass": out["mass"]}


def _own_evict(s):
    sv, h = _handle()
    case = s["case"]
    out = sv.specv_cache_evict(h, s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["mass"], case["budget"],
                               recent=case["recent"], first=case["first"], out=s["out"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "mass": out["mass"], "seq_lens": out["seq_lens"],
            "evicted": out["evicted"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "prefix": _own_prefix, "mass": _own_mass, "evict": _own_evict}[op](state)
    return {"append": _plain_append, "prefix": _plain_prefix, "mass": _plain_mass, "evict": _plain_evict}[op](state)


# ---------------------------------------------------------------------------- the least work
def work(case):
    """Bytes and operations at the mean of the ragged lengths."""
    size = 2 if case["dtype"] == "bf16" else 4
    batch, heads, dim = case["batch"], case["kv_heads"], case["head_dim"]
    if case["op"] == "evict":
        budget, recent, first = case["budget"], case["recent"], case["first"]
        mean = (budget + recent + case["length"]) / 2
        many = 1 + (batch - 1) * 0.9  # sequences over the budget
        kept = budget - recent - first
        beyond = mean - budget - recent  # candidates above the line that may be kept
        moved = recent + kept * max(0.0, beyond) / max(1.0, kept + beyond)
        rows = many * heads * case["layers"]
        return {"bytes": rows * (moved * dim * size * 4 + (mean + budget) * 4), "flops": 0}
    rows, q_heads = case["rows"], case["q_heads"]
    if case["op"] == "append":
        tokens = rows * batch if not case["ragged"] else rows + (batch - 1) * (rows + 1) / 2
        ops = 3 * case["rot"] + (4 * dim if case["norm"] else 0)
        return {"bytes": tokens * dim * size * (2 * q_heads + 4 * heads) + (batch * rows - tokens) * q_heads * dim * size
                + tokens * 4 * case["axes"],
                "flops": tokens * (q_heads + heads) * ops}
    low = max(rows, case["length"] // 2)
    keys = max(rows, case["length"]) + (batch - 1) * (low + max(rows, case["length"])) / 2
    pairs = rows * (keys - batch * rows / 2)
    if case["op"] == "mass":
        scored = max(1.0, keys - batch * case["first"])
        return {"bytes": scored * heads * (dim * size + (4 if case["start"] else 8))
                + batch * rows * q_heads * (dim * size + 4),
                "flops": 2 * q_heads * dim * rows * scored}
    return {"bytes": 2 * (keys + case["prefix"]) * heads * dim * size + 2 * batch * rows * q_heads * dim * size,
            "flops": 4 * q_heads * dim * (pairs + batch * rows * case["prefix"])}


# ---------------------------------------------------------------------------- 64 bits
def _depths_and_masks(parents, rows):
    """Of one sequence: the depth of every row, and the rows it may see."""
    depth, seen = [0], [{0}]
    for i in range(rows - 1):
        p = (i - 1 if parents is None else int(parents[i])) + 1
        depth.append(depth[p] + 1)
        seen.append(seen[p] | {i + 1})
    return depth, seen


def _unit(x, weight):
    """x [n, H, D] in 64 bits over its root of the mean square, times the weight."""
    x = x.double()
    if weight is None:
        return x
    return x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * weight.double()


def _turned(x, angle, interleaved):
    """x [n, H, D] in 64 bits with its pairs turned as complex numbers by angle [n, pairs]."""
    x = x.clone()
    r = 2 * angle.shape[1]
    first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous())
    angle = angle[:, None]
    z = z * torch.polar(torch.ones_like(angle), angle)
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_append(case, s):
    bs, lens, tables, rows = case["block_size"], s["lens"].tolist(), s["tables"].long(), case["rows"]
    q, k, v = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), s["k_cache"].double(), s["v_cache"].double()
    parents = None if s["parents"] is None else s["parents"].tolist()
    counts = [rows] * len(lens) if s["counts"] is None else s["counts"].tolist()
    shift = [0] * len(lens) if s["offsets"] is None else s["offsets"].tolist()
    freq = s["inv_freq"].double()
    for b, (n, m) in enumerate(zip(lens, counts)):
        if s["positions"] is None:
            depth = list(range(m)) if parents is None else _depths_and_masks(parents[b], rows)[0][:m]
            pos = torch.tensor(depth, dtype=torch.float64, device="cuda") + (n - m + shift[b])
            angle = torch.outer(pos, freq)
        else:
            angle = torch.stack([s["positions"][b, :m, a].double() * freq[j] for j, a in enumerate(s["axis"])], -1)
        slot = torch.arange(n - m, n, device="cuda")
        q[b, :m] = _turned(_unit(s["q"][b, :m], s["q_norm"]), angle, case["interleaved"])
        k[tables[b, slot // bs], :, slot % bs] = _turned(_unit(s["k"][b, :m], s["k_norm"]), angle, case["interleaved"])
        v[tables[b, slot // bs], :, slot % bs] = s["v"][b, :m].double()
    return {"q": q, "k_cache": k, "v_cache": v}


def _exact_rows(case, s, b, n):
    """Scores [heads, group, rows, n] of sequence b in 64 bits, -inf where a row does not see a position; its blocks and
    places."""
    bs, rows = case["block_size"], case["rows"]
    _, seen = _depths_and_masks(None if s["parents"] is None else s["parents"][b].tolist(), rows)
    shut = torch.zeros((rows, n), dtype=torch.bool)
    for r in range(rows):
        shut[r, [n - rows + j for j in range(rows) if j not in seen[r]]] = True
    slot = torch.arange(n, device="cuda")
    block = s["tables"][b].long()[slot // bs]
    k = s["k_cache"][block, :, slot % bs].double()
    q = s["q"][b].double().reshape(rows, case["kv_heads"], -1, case["head_dim"])
    x = torch.einsum("rhgd,nhd->hgrn", q, k) / math.sqrt(case["head_dim"])
    return x.masked_fill(shut.cuda(), -math.inf), block, slot % bs


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    lens = s["lens"].tolist()
    if case["op"] == "evict":
        k, v, mass = s["k_cache"].double(), s["v_cache"].double(), s["out"]["mass"].double()
        budget, recent, first, bs = case["budget"], case["recent"], case["first"], case["block_size"]
        many = budget - recent - first
        seen = s["mass"].cpu()
        for b, n in enumerate(lens):
            if n <= budget:
                mass[:, b, :, :n] = s["mass"][:, b, :, :n].double()
                continue
            block = s["tables"][b].long()
            for l in range(case["layers"]):
                for h in range(case["kv_heads"]):
                    row = seen[l, b, h, first:n - recent].tolist()
                    best = sorted(range(len(row)), key=lambda i: (-row[i], i))[:many]
                    late = sorted(i for i in best if i >= many)
                    free = sorted(set(range(many)) - set(best))
                    place = list(range(n))  # which position ends up where
                    for i, j in zip(free, late):
                        place[first + i] = first + j
                    place[first + many:budget] = range(n - recent, n)
                    to = torch.tensor([i for i in range(budget) if place[i] != i], dtype=torch.int64, device="cuda")
                    src = torch.tensor(place[:budget], dtype=torch.int64, device="cuda")
                    mass[l, b, h, :budget] = s["mass"][l, b, h, src].double()
                    src = src[to]
                    for x in (k, v):
                        x[l, block[to // bs], h, to % bs] = x[l, block[src // bs], h, src % bs]
        ends = torch.tensor([min(n, budget) for n in lens], device="cuda")
        return {"k_cache": k, "v_cache": v, "mass": mass, "seq_lens": ends, "evicted": s["lens"] - ends}
    rows, heads, dim = case["rows"], case["kv_heads"], case["head_dim"]
    if case["op"] == "mass":
        out = s["out"]["mass"].double()
        for b, n in enumerate(lens):
            x, _, _ = _exact_rows(case, s, b, n)
            lse = s["lse"][b].double().reshape(rows, heads, -1).permute(1, 2, 0)
            got = (x - lse[..., None]).exp().sum((1, 2))
            if s["mass"] is not None:
                got[:, :n - rows] += s["mass"][b, :, :n - rows].double()
            out[b, :, case["first"]:n] = got[:, case["first"]:]
        return {"mass": out}
    outs, sums = [], []
    for b, n in enumerate(lens):
        x, block, place = _exact_rows(case, s, b, n)
        v = s["v_cache"][block, :, place].double()
        sums.append(torch.logsumexp(x, -1).permute(2, 0, 1).reshape(rows, -1))
        outs.append(torch.einsum("hgrn,nhd->rhgd", torch.softmax(x, -1), v).reshape(rows, -1, dim))
    got = {"out": torch.stack(outs)}
    if case["lse"]:
        got["lse"] = torch.stack(sums)
    return got
