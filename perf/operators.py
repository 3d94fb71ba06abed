"""Cases for the operators on the paged KV cache: append with rotation, attention for
draft trees, compaction of the kept path.

A cache is a pool of blocks [blocks, kv_heads, block_size, head_dim] for keys and one
for values; row b of the block table names the blocks of sequence b, and seq_lens[b] is
the number of positions it holds, the rows of the current pass the last of them (as
specv_rollback counts them).  Row 0 of a pass is the token after the verified prefix,
row 1 + i is draft node i; parents[i] is a node, or -1 for a child of row 0.
"""
import functools
import math

import torch

own = False


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of a few sequences: a decode step without drafts
        dict(name="append token", op="append", dtype="bf16", batch=8, rows=1, tree=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, rot=128, interleaved=False, length=2000, ragged=False),
        # a draft tree for every sequence of a serving batch
        dict(name="append tree", op="append", dtype="bf16", batch=64, rows=17, tree=True, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, rot=128, interleaved=False, length=1000, ragged=False),
        # ragged prompts, padded to the longest, on top of a cached prefix
        dict(name="append prompt", op="append", dtype="bf16", batch=4, rows=2048, tree=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, rot=128, interleaved=False, length=500, ragged=True),
        # a small fp32 draft model: chains of 4, half of the head rotated, interleaved pairs
        dict(name="append f32", op="append", dtype="f32", batch=16, rows=5, tree=False, q_heads=12, kv_heads=12,
             head_dim=64, block_size=16, rot=32, interleaved=True, length=700, ragged=False),
        # a decode step: one row a sequence
        dict(name="attend token", op="attend", dtype="bf16", batch=8, rows=1, tree=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, length=1000, lse=False),
        # chains of 5 drafts in a serving batch
        dict(name="attend chain", op="attend", dtype="bf16", batch=64, rows=6, tree=False, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, length=2000, lse=False),
        # trees of 16 nodes in the same batch, longer contexts
        dict(name="attend tree", op="attend", dtype="bf16", batch=64, rows=17, tree=True, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, length=4096, lse=False),
        # the widest trees, eight query heads to a kv head
        dict(name="attend wide tree", op="attend", dtype="bf16", batch=16, rows=32, tree=True, q_heads=64, kv_heads=8,
             head_dim=128, block_size=32, length=8192, lse=True),
        # one user with a very long context
        dict(name="attend long", op="attend", dtype="bf16", batch=1, rows=17, tree=True, q_heads=32, kv_heads=8,
             head_dim=128, block_size=16, length=131072, lse=True),
        # the fp32 draft model
        dict(name="attend f32", op="attend", dtype="f32", batch=8, rows=5, tree=False, q_heads=12, kv_heads=12,
             head_dim=64, block_size=16, length=1000, lse=False),
        # one layer of a small batch after verification
        dict(name="compact layer", op="compact", dtype="bf16", batch=8, nodes=6, layers=1, kv_heads=8, head_dim=128,
             block_size=16, length=200),
        # all layers of a serving batch
        dict(name="compact layers", op="compact", dtype="bf16", batch=64, nodes=16, layers=32, kv_heads=8,
             head_dim=128, block_size=16, length=60),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    c = dict(op=op, dtype=dtype, batch=_spread(rng, 1, 128), kv_heads=rng.choice([1, 2, 4, 8, 10]),
             head_dim=rng.choice([64, 64, 96, 128, 128, 128, 256]), block_size=rng.choice([5, 8, 16, 16, 16, 32, 64]))
    line = c["kv_heads"] * c["head_dim"] * size  # bytes of one position of one cache
    if op == "compact":
        c["nodes"] = rng.randint(1, 31)
        c["length"] = _spread(rng, c["nodes"] + 1, 300)
        blocks = c["batch"] * (c["length"] // c["block_size"] + 2)
        c["layers"] = _spread(rng, 1, max(1, min(48, int(6e8 / (blocks * c["block_size"] * line)))))
        return c
    c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 3, 4, 4, 5, 8])
    c["tree"] = rng.random() < 0.6
    if op == "append":
        c["rows"] = rng.randint(1, 32) if c["tree"] else _spread(rng, 1, 2048)
        tokens = int(1.2e8 / (line * (1 + c["q_heads"] // c["kv_heads"])))
        c["batch"] = max(1, min(c["batch"], tokens // c["rows"], int(2.5e8 / (1200 * line))))
        c["rows"] = min(c["rows"], tokens)
        c["rot"] = rng.choice([c["head_dim"], c["head_dim"], c["head_dim"] // 2, 0])
        c["interleaved"] = rng.random() < 0.3
        c["ragged"] = not c["tree"] and rng.random() < 0.7
        c["length"] = c["rows"] + _spread(rng, 1, 1000)
        return c
    c["rows"] = rng.randint(1, 32)
    # no more bytes, and no more products, than the largest listed cases
    keys = min(5e8 / (2 * line), 3e10 / (4 * c["rows"] * c["q_heads"] * c["head_dim"]))
    if dtype == "f32":
        keys /= 4
    c["length"] = _spread(rng, c["rows"], max(c["rows"], min(131072, int(keys))))
    c["batch"] = max(1, min(c["batch"], int(keys / c["length"])))
    c["lse"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------- inputs
def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _pool(shape, dtype, g):
    """A pool of keys or values, leftovers of earlier sequences in the positions that none holds."""
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def _tables(lens, block_size, g):
    """Blocks for sequences of these lengths, shuffled over a pool with some to spare; -1 behind the last."""
    used = [(n + block_size - 1) // block_size for n in lens]
    total = len(lens) * max(used) + 7
    order = torch.randperm(total, generator=g)
    table = torch.full((len(lens), max(used)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.Generator().manual_seed(seed)
    dtype, batch = _type(case), case["batch"]
    heads, dim, bs = case["kv_heads"], case["head_dim"], case["block_size"]
    s = dict(case=case)
    if case["op"] == "compact":
        # breadth-first trees; the kept path takes a node of each level.  No slot that is written is read too, so
        # that a pass can be repeated on the same caches: the first level keeps its first node or a late one.
        nodes = case["nodes"]
        width = math.isqrt(nodes - 1) + 1
        depth = nodes // width
        kept = torch.randint(0, depth + 1, (batch,), generator=c)
        kept[0] = depth
        level = torch.arange(nodes)
        pick = torch.floor(torch.rand((batch, nodes), generator=c) * width).to(torch.int64)
        path = level * width + pick
        first = torch.where(pick[:, 0] >= kept, pick[:, 0], 0)
        path[:, 0] = first
        path = torch.where(level < kept[:, None], path, -1)
        lens = _lengths(case, nodes + 1, c)
        s["tables"], total = _tables(lens.tolist(), bs, c)
        s["k_cache"] = _pool((case["layers"], total, heads, bs, dim), dtype, g)
        s["v_cache"] = _pool((case["layers"], total, heads, bs, dim), dtype, g)
        s["path"], s["kept"] = path.to(torch.int32).cuda(), kept.to(torch.int32).cuda()
        s["lens"] = lens.to(torch.int32).cuda()
        s["status"] = torch.empty(batch, dtype=torch.int32, device="cuda")
        return s
    rows, q_heads = case["rows"], case["q_heads"]
    s["parents"] = _random_parents(batch, rows - 1, c).cuda() if case["tree"] else None
    lens = _lengths(case, rows, c)
    if case["op"] == "append":
        s["counts"] = None
        if case["ragged"]:
            counts = torch.randint(1, rows + 1, (batch,), generator=c)
            counts[0] = rows
            lens = lens - rows + counts
            s["counts"] = counts.to(torch.int32).cuda()
        s["inv_freq"] = None
        if case["rot"]:
            s["inv_freq"] = (10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])).float().cuda()
    s["tables"], total = _tables(lens.tolist(), bs, c)
    s["lens"] = lens.to(torch.int32).cuda()
    s["k_cache"] = _pool((total, heads, bs, dim), dtype, g)
    s["v_cache"] = _pool((total, heads, bs, dim), dtype, g)
    # queries, keys and values lie behind one another, as one product of the hidden state gives them
    fused = torch.randn((batch, rows, q_heads + 2 * heads, dim), generator=g, device="cuda")
    fused[:, :, :q_heads] *= 2  # scores that spread by two: a few positions of a context carry most of the weight
    fused = fused.to(dtype)
    s["q"], s["k"], s["v"] = fused[:, :, :q_heads], fused[:, :, q_heads:q_heads + heads], fused[:, :, q_heads + heads:]
    s["out"] = {"row_status": torch.empty(batch, dtype=torch.int32, device="cuda"),
                "q_out" if case["op"] == "append" else "out":
                torch.empty((batch, rows, q_heads, dim), dtype=dtype, device="cuda")}
    if case["op"] == "attend" and case["lse"]:
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


def _rotate(x, pos, inv_freq, interleaved):
    """x [B, R, H, D] rotated in its first 2 len(inv_freq) values by pos [B, R]."""
    if inv_freq is None:
        return x.float()
    half = inv_freq.numel()
    angle = pos.double()[:, :, None] * inv_freq.double()
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    x, rest = x[..., :2 * half].float(), x[..., 2 * half:].float()
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
    depth = at.expand(batch, rows) if s["parents"] is None else _reach(s["parents"], batch, rows).sum(-1) - 1
    pos = base[:, None] + depth
    real = at < counts[:, None]
    q = _rotate(s["q"], pos, s["inv_freq"], case["interleaved"]).to(dtype)
    q = torch.where(real[:, :, None, None], q, torch.zeros((), dtype=dtype, device="cuda"))
    k = _rotate(s["k"], pos, s["inv_freq"], case["interleaved"]).to(dtype)
    # rows behind a sequence's last write what its row 0 writes, once more
    row = torch.where(real, at, 0)
    slot = base[:, None] + row
    block = s["tables"].long().gather(1, slot // bs)
    pick = row[:, :, None, None]
    s["k_cache"][block, :, slot % bs] = torch.take_along_dim(k, pick, 1)
    s["v_cache"][block, :, slot % bs] = torch.take_along_dim(s["v"], pick, 1)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    case, bs = s["case"], s["case"]["block_size"]
    batch, rows, heads, dim = case["batch"], case["rows"], case["kv_heads"], case["head_dim"]
    group = case["q_heads"] // heads
    table = s["tables"].long().clamp(min=0)
    n = table.shape[1] * bs
    k = s["k_cache"][table].transpose(1, 2).reshape(batch, heads, n, dim).float()
    v = s["v_cache"][table].transpose(1, 2).reshape(batch, heads, n, dim).float()
    q = s["q"].float().reshape(batch, rows, heads, group, dim).permute(0, 2, 1, 3, 4).reshape(batch, heads, -1, dim)
    # slots before the pass's rows are open to each of them, the pass's own by the tree
    node = torch.arange(n, device="cuda") - (s["lens"].long() - rows)[:, None]
    seen = _reach(s["parents"], batch, rows).gather(2, node.clamp(0, rows - 1)[:, None].expand(batch, rows, n))
    seen = (node < 0)[:, None] | (seen & (node < rows)[:, None])
    x = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(dim)).view(batch, heads, rows, group, n)
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(batch, heads, rows * group, n) @ v).view(batch, heads, rows, group, dim) / total
    got = {"out": o.permute(0, 2, 1, 3, 4).reshape(batch, rows, heads * group, dim).to(s["q"].dtype)}
    if case["lse"]:
        got["lse"] = (top + total.log()).view(batch, heads, rows, group).permute(0, 2, 1, 3).reshape(batch, rows, -1)
    return got


def _plain_compact(s):
    bs, nodes = s["case"]["block_size"], s["case"]["nodes"]
    base = (s["lens"].long() - nodes)[:, None]
    to = torch.arange(nodes, device="cuda")
    # behind the kept path every node stays where it is
    src = base + torch.where(to < s["kept"][:, None], s["path"].long(), to)
    # a node that another one is moved from keeps its own value: the path's slots are read before any is written
    dst = base + to
    table = s["tables"].long()
    a, b = table.gather(1, src // bs), table.gather(1, dst // bs)
    s["k_cache"][:, b, :, dst % bs] = s["k_cache"][:, a, :, src % bs]
    s["v_cache"][:, b, :, dst % bs] = s["v_cache"][:, a, :, src % bs]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ---------------------------------------------------------------------------- the framework's calls
@functools.lru_cache(maxsize=None)
def _handle():
    import speculative_decoding_verification_57_gb300 as sv

    return sv, sv.specv_create(0, max_batch=256, max_k=31)


def _own_append(s):
    sv, h = _handle()
    out = sv.specv_cache_append(h, s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["k"], s["v"], q=s["q"],
                                inv_freq=s["inv_freq"], interleaved=s["case"]["interleaved"], parents=s["parents"],
                                row_counts=s["counts"], out=s["out"])
    return {"q": out["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    sv, h = _handle()
    out = sv.specv_tree_attention(h, s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], parents=s["parents"],
                                  lse=s["case"]["lse"], out=s["out"])
    return {"out": out["out"], "lse": out["lse"]} if s["case"]["lse"] else {"out": out["out"]}


def _own_compact(s):
    sv, h = _handle()
    sv.specv_cache_compact(h, s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["path"], s["kept"],
                           row_status=s["status"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "compact": _own_compact}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "compact": _plain_compact}[op](state)


# ---------------------------------------------------------------------------- the least work
def work(case):
    """Bytes and operations at the mean of the ragged lengths."""
    size = 2 if case["dtype"] == "bf16" else 4
    batch, heads, dim = case["batch"], case["kv_heads"], case["head_dim"]
    if case["op"] == "compact":
        depth = case["nodes"] // (math.isqrt(case["nodes"] - 1) + 1)
        moved = max(1.0, (depth + (batch - 1) * depth / 2)) * case["layers"]
        return {"bytes": moved * heads * dim * size * 2 * 2, "flops": 0}
    rows, q_heads = case["rows"], case["q_heads"]
    if case["op"] == "append":
        tokens = rows * batch if not case["ragged"] else rows + (batch - 1) * (rows + 1) / 2
        return {"bytes": tokens * dim * size * (2 * q_heads + 4 * heads) + (batch * rows - tokens) * q_heads * dim * size,
                "flops": 3 * tokens * (q_heads + heads) * case["rot"]}
    low = max(rows, case["length"] // 2)
    keys = max(rows, case["length"]) + (batch - 1) * (low + max(rows, case["length"])) / 2
    pairs = rows * (keys - batch * rows / 2)
    return {"bytes": 2 * keys * heads * dim * size + 2 * batch * rows * q_heads * dim * size,
            "flops": 4 * q_heads * dim * pairs}


# ---------------------------------------------------------------------------- 64 bits
def _depths_and_masks(parents, rows):
    """Of one sequence: the depth of every row, and the rows it may see."""
    depth, seen = [0], [{0}]
    for i in range(rows - 1):
        p = (i - 1 if parents is None else int(parents[i])) + 1
        depth.append(depth[p] + 1)
        seen.append(seen[p] | {i + 1})
    return depth, seen


def _turned(x, pos, inv_freq, interleaved):
    """x [n, H, D] in 64 bits with its pairs turned as complex numbers."""
    x = x.double().clone()
    if inv_freq is None:
        return x
    r = 2 * inv_freq.numel()
    first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous())
    angle = torch.outer(pos, inv_freq.double())[:, None]
    z = z * torch.polar(torch.ones_like(angle), angle)
    x[..., first], x[..., second] = z.real, z.imag
    return x


def exact(case, seed):
    s = prepare(case, seed)
    bs, lens, tables = case["block_size"], s["lens"].tolist(), s["tables"].long()
    if case["op"] == "compact":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        for b, n in enumerate(lens):
            base = n - case["nodes"]
            for i in range(int(s["kept"][b])):
                src, dst = base + int(s["path"][b, i]), base + i
                for x in (k, v):
                    x[:, tables[b, dst // bs], :, dst % bs] = x[:, tables[b, src // bs], :, src % bs]
        return {"k_cache": k, "v_cache": v}
    rows = case["rows"]
    if case["op"] == "append":
        q, k, v = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), s["k_cache"].double(), s["v_cache"].double()
        parents = None if s["parents"] is None else s["parents"].tolist()
        counts = [rows] * len(lens) if s["counts"] is None else s["counts"].tolist()
        for b, (n, m) in enumerate(zip(lens, counts)):
            base = n - m
            depth = list(range(m)) if parents is None else _depths_and_masks(parents[b], rows)[0][:m]
            pos = torch.tensor(depth, dtype=torch.float64, device="cuda") + base
            slot = torch.arange(base, n, device="cuda")
            q[b, :m] = _turned(s["q"][b, :m], pos, s["inv_freq"], case["interleaved"])
            k[tables[b, slot // bs], :, slot % bs] = _turned(s["k"][b, :m], pos, s["inv_freq"], case["interleaved"])
            v[tables[b, slot // bs], :, slot % bs] = s["v"][b, :m].double()
        return {"q": q, "k_cache": k, "v_cache": v}
    heads, dim, group = case["kv_heads"], case["head_dim"], case["q_heads"] // case["kv_heads"]
    parents = None if s["parents"] is None else s["parents"].tolist()
    outs, sums = [], []
    for b, n in enumerate(lens):
        _, seen = _depths_and_masks(None if parents is None else parents[b], rows)
        shut = torch.zeros((rows, n), dtype=torch.bool)
        for r in range(rows):
            shut[r, [n - rows + j for j in range(rows) if j not in seen[r]]] = True
        slot = torch.arange(n, device="cuda")
        k = s["k_cache"][tables[b, slot // bs], :, slot % bs].double()
        v = s["v_cache"][tables[b, slot // bs], :, slot % bs].double()
        q = s["q"][b].double().reshape(rows, heads, group, dim)
        x = torch.einsum("rhgd,nhd->hgrn", q, k) / math.sqrt(dim)
        x = x.masked_fill(shut.cuda(), -math.inf)
        sums.append(torch.logsumexp(x, -1).permute(2, 0, 1).reshape(rows, -1))
        outs.append(torch.einsum("hgrn,nhd->rhgd", torch.softmax(x, -1), v).reshape(rows, -1, dim))
    got = {"out": torch.stack(outs)}
    if case["lse"]:
        got["lse"] = torch.stack(sums)
    return got
