"""GPU parity of the calls on the paged KV cache with their plain float64
restatements (cache_plain.py): append with rotation, attention for draft
trees, compaction of the kept path, and a verify round made of them."""
import math

import numpy as np
import pytest

import cache_plain as P

pytestmark = pytest.mark.gpu

BF16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_57_gb300 as sv

    return sv


@pytest.fixture(scope="module")
def h(sv):
    handle = sv.specv_create(0, max_batch=512, max_k=31, vocab=1000)
    yield handle
    sv.specv_destroy(handle)


def _dtype(name):
    import torch

    return torch.bfloat16 if name == "bf16" else torch.float32


def _dev(a, dtype=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def _np(t):
    return t.detach().double().cpu().numpy()


def _rounded(rng, shape, dtype, scale=1.0):
    """Normal values that the type holds exactly: (device tensor, float64 array)."""
    import torch

    t = torch.from_numpy(rng.normal(scale=scale, size=shape).astype(np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def _random_tree(rng, kind, B, rows):
    if rows == 1:
        return None if kind == "chain" else np.zeros((B, 0), np.int32)
    if kind == "chain":
        return None
    if kind == "star":
        return np.full((B, rows - 1), -1, np.int32)
    if kind == "line":
        return np.tile(np.arange(-1, rows - 2, dtype=np.int32), (B, 1))
    return np.array([[rng.integers(-1, i) for i in range(rows - 1)] for _ in range(B)], np.int32)


def _tables(rng, lens, bs, width=None, spare=3):
    """Shuffled blocks for these lengths, -1 behind the last; (tables, blocks)."""
    used = [-(-int(n) // bs) for n in lens]
    width = max(used + [1]) if width is None else width
    order = rng.permutation(sum(used) + spare)
    tables = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(used):
        tables[b, :n] = order[at:at + n]
        at += n
    return tables, sum(used) + spare


class Case:
    """Inputs of an attention call; positions that no sequence holds are NaN."""

    def __init__(self, seed, dtype, B, rows, hq, hkv, dim, bs, lens, kind="tree", q_scale=1.5, poison=True, width=None):
        import torch

        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.rows = rng, _dtype(dtype), rows
        self.lens = np.array(lens, np.int32)
        assert len(lens) == B
        self.tables, blocks = _tables(rng, np.maximum(self.lens, 0), bs, width)
        self.kc_t, self.kc = _rounded(rng, (blocks, hkv, bs, dim), self.dtype)
        self.vc_t, self.vc = _rounded(rng, (blocks, hkv, bs, dim), self.dtype)
        if poison:
            held = np.zeros((blocks, bs), bool)
            for b, n in enumerate(self.lens):
                t = np.arange(max(int(n), 0))
                held[self.tables[b, t // bs], t % bs] = True
            hole = torch.from_numpy(~held).cuda()[:, None, :, None]
            self.kc_t.masked_fill_(hole, math.nan)
            self.vc_t.masked_fill_(hole, math.nan)
        self.q_t, self.q = _rounded(rng, (B, rows, hq, dim), self.dtype, q_scale)
        self.parents = _random_tree(rng, kind, B, rows)
        self.scale = dim ** -0.5
        self.ref = None  # of the first check; the inputs stay from then on

    def call(self, sv, h, **kw):
        import torch

        par = None if self.parents is None else _dev(self.parents)
        got = sv.specv_tree_attention(h, kw.pop("q", self.q_t), self.kc_t, self.vc_t, _dev(self.tables),
                                      _dev(self.lens), parents=par, lse=True, **kw)
        torch.cuda.synchronize()
        return got

    def check(self, got, scale=None):
        scale = self.scale if scale is None else scale
        if self.ref is None or self.ref[0] != scale:
            self.ref = scale, P.attention(self.q, _np(self.kc_t), _np(self.vc_t), self.tables, self.lens, self.parents,
                                          scale)
        out, lse, status, avg, mag = self.ref[1]
        np.testing.assert_array_equal(got["row_status"].cpu().numpy(), status)
        g, gl = _np(got["out"]), _np(got["lse"])
        same = np.isfinite(out)
        np.testing.assert_array_equal(np.isnan(g), np.isnan(out))
        np.testing.assert_array_equal(g[np.isinf(out)], out[np.isinf(out)])
        n_max = int(max(self.lens.max(), 1))
        t_out, t_lse = P.attention_bounds(out, np.where(np.isfinite(lse), lse, 0), avg, mag, n_max, self.q.shape[-1],
                                          str(self.dtype).endswith("bfloat16"))
        bad = same & ~(np.abs(g - np.where(same, out, 0)) <= t_out)
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], g[bad][:4], out[bad][:4], t_out[bad][:4])
        fin = np.isfinite(lse)
        np.testing.assert_array_equal(gl[~fin], lse[~fin])
        bad = fin & ~(np.abs(gl - np.where(fin, lse, 0)) <= t_lse)
        assert not bad.any(), (gl[bad][:4], lse[bad][:4], t_lse[bad][:4])


# ---------------------------------------------------------------------------- attention
SHAPES = [
    # B, rows, q heads, kv heads, dim, block, lengths, tree
    (1, 1, 1, 1, 16, 1, [1], "chain"),
    (1, 1, 4, 2, 64, 16, [1], "tree"),
    (3, 1, 8, 2, 128, 16, [16, 17, 400], "chain"),
    (4, 1, 32, 8, 128, 16, [0, 1, 63, 64], "chain"),
    (5, 3, 6, 2, 80, 5, [3, 0, 64, 65, 131], "tree"),
    (2, 2, 8, 1, 64, 7, [2, 129], "star"),
    (4, 6, 8, 2, 128, 16, [6, 127, 128, 300], "chain"),
    (4, 17, 8, 2, 128, 16, [17, 33, 128, 257], "tree"),
    (2, 17, 16, 2, 96, 32, [40, 200], "tree"),
    (2, 32, 8, 1, 128, 16, [32, 290], "tree"),
    (2, 32, 16, 2, 128, 64, [33, 500], "line"),
    (2, 32, 12, 4, 64, 16, [64, 321], "star"),
    (2, 9, 24, 1, 256, 16, [9, 150], "tree"),
    (1, 32, 40, 1, 256, 8, [260], "tree"),
    (3, 31, 5, 5, 48, 3, [31, 95, 96], "tree"),
    (7, 4, 10, 10, 64, 16, [4, 20, 0, 100, 64, 63, 5], "tree"),
    # more than 16 rows a kv head: every way blocks and queries come to the tensor cores
    (3, 20, 4, 2, 16, 16, [20, 130, 300], "tree"),
    (3, 20, 6, 2, 48, 8, [21, 128, 260], "tree"),
    (2, 24, 10, 2, 80, 64, [24, 200], "star"),
    (2, 18, 14, 2, 112, 128, [130, 270], "tree"),
    (2, 32, 16, 2, 128, 256, [255, 600], "tree"),
    (2, 32, 16, 2, 64, 24, [96, 420], "tree"),
    (1, 32, 40, 1, 128, 16, [300], "tree"),
    (2, 32, 24, 1, 64, 1, [32, 135], "line"),
    (2, 1, 64, 1, 128, 16, [1, 700], "chain"),
    (3, 11, 12, 6, 128, 16, [0, 128, 129], "chain"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%d_R%d_H%d-%d_D%d_bs%d_%s" % (s[:6] + (s[7],)))
def test_attention_matches_the_formula(sv, h, dtype, shape):
    B, rows, hq, hkv, dim, bs, lens, kind = shape
    c = Case(B * 1000 + rows * 10 + dim, dtype, B, rows, hq, hkv, dim, bs, lens, kind)
    c.check(c.call(sv, h))


@pytest.mark.parametrize("dtype,rows,hq,hkv,length", [("bf16", 1, 4, 1, 20011), ("bf16", 17, 4, 1, 9001),
                                                      ("bf16", 32, 8, 1, 5003), ("f32", 3, 2, 1, 7001)])
def test_attention_over_a_long_cache(sv, h, dtype, rows, hq, hkv, length):
    c = Case(rows, dtype, 2, rows, hq, hkv, 128, 16, [length, 77], "tree")
    c.check(c.call(sv, h))


def test_attention_of_many_sequences(sv, h):
    rng = np.random.default_rng(5)
    lens = rng.integers(3, 200, size=150)
    lens[::13] = 0
    c = Case(6, "bf16", 150, 3, 8, 4, 64, 16, lens, "tree")
    c.check(c.call(sv, h))


def test_attention_of_more_sequences_than_threads(sv):
    """The cut of the work goes over the lengths in several passes."""
    rng = np.random.default_rng(7)
    handle = sv.specv_create(0, max_batch=2000, max_k=31, vocab=1000)
    for dtype, rows, B in (("bf16", 9, 1100), ("f32", 1, 700), ("bf16", 1, 1300)):
        lens = rng.integers(rows, 40, size=B)
        lens[::17] = 0
        lens[5], lens[B - 2] = 500, 700
        c = Case(B, dtype, B, rows, 2, 1, 16, 16, lens, "tree")
        c.check(c.call(sv, handle))
    sv.specv_destroy(handle)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hq", [(2, 2), (7, 8), (32, 8)])
def test_rows_do_not_see_what_the_tree_hides(sv, h, dtype, rows, hq):
    """NaN and infinities in the keys and values of other branches leave a row
    as it is; its own and its ancestors' come through."""
    c = Case(rows, dtype, 3, rows, hq, 1, 64, 16, [rows, rows + 30, 200], "star")
    nan, inf = math.nan, math.inf
    for b, (bk, bv) in enumerate([(nan, nan), (0.0, inf), (nan, -inf)]):
        t = int(c.lens[b]) - 1  # the last node: seen by itself alone
        blk, slot = int(c.tables[b, t // 16]), t % 16
        if bk != 0.0:
            c.kc_t[blk, :, slot, 3] = bk
        c.vc_t[blk, :, slot, 5] = bv
    got = c.call(sv, h)
    c.check(got)
    g = _np(got["out"])
    assert np.isfinite(g[:, :rows - 1]).all() and not np.isfinite(g[:, rows - 1]).all()


def test_values_of_a_hidden_branch_at_the_ends_of_the_type(sv, h):
    import torch

    c = Case(3, "bf16", 1, 20, 4, 1, 128, 16, [150], "tree")
    big = torch.finfo(torch.bfloat16).max
    for node, val in ((4, big), (9, -big), (19, math.inf)):
        t = 130 + node
        c.vc_t[int(c.tables[0, t // 16]), :, t % 16, node:node + 3] = val
    c.check(c.call(sv, h))


def test_large_scores_and_a_negative_scale(sv, h):
    c = Case(4, "bf16", 2, 5, 4, 2, 64, 16, [100, 9], "tree", q_scale=60.0)
    c.check(c.call(sv, h))
    c = Case(5, "f32", 2, 5, 4, 2, 64, 16, [100, 9], "tree")
    c.check(c.call(sv, h, scale=-0.7), scale=-0.7)
    c.check(c.call(sv, h, scale=0.0), scale=0.0)


@pytest.mark.parametrize("rows,hq", [(17, 8), (32, 16)])
def test_scales_and_large_scores_with_many_rows(sv, h, rows, hq):
    c = Case(4, "bf16", 2, rows, hq, 2, 128, 16, [300, rows + 2], "tree", q_scale=60.0)
    c.check(c.call(sv, h))
    c = Case(5, "bf16", 2, rows, hq, 2, 64, 16, [300, rows + 2], "tree")
    c.check(c.call(sv, h, scale=-0.7), scale=-0.7)
    c.check(c.call(sv, h, scale=0.0), scale=0.0)
    c.check(c.call(sv, h, scale=3.0), scale=3.0)


@pytest.mark.parametrize("rows,hq", [(3, 4), (17, 8), (32, 16)])
def test_not_finite_queries_and_prefix(sv, h, rows, hq):
    """Of a query that is not finite its own row alone is; a key or value that
    every row sees reaches them all."""
    c = Case(6, "bf16", 3, rows, hq, 2, 128, 16, [200, 150, rows], "tree")
    c.q_t[0, 1, 0, 7] = math.nan
    c.q[0, 1, 0, 7] = math.nan
    c.vc_t[int(c.tables[1, 2]), 1, 5, 3] = math.inf  # position 37 of sequence 1
    got = c.call(sv, h)
    c.check(got)
    g = _np(got["out"])
    assert np.isnan(g[0, 1, 0]).all() and np.isnan(g[0]).sum() == 128
    assert np.isinf(g[1][:, hq // 2:, 3]).all() and np.isfinite(g[2]).all()


@pytest.mark.parametrize("rows,hq,bs", [(3, 4, 16), (17, 8, 16), (17, 8, 6), (32, 16, 16)])
def test_many_segments_a_cta_and_holes(sv, bs, rows, hq):
    """Hundreds of short sequences, so that a CTA goes through many segments,
    some with blocks outside the pool: only these are refused."""
    rng = np.random.default_rng(rows)
    handle = sv.specv_create(0, max_batch=2000, max_k=31, vocab=1000)
    B = 900 if rows < 30 else 700
    lens = rng.integers(rows, rows + 60, size=B)
    lens[::9] = 0
    c = Case(rows, "bf16", B, rows, hq, hq // 2 if rows < 17 else 4, 16, bs, lens, "tree")
    for b in range(0, B, 31):
        if c.lens[b]:
            c.tables[b, rng.integers(0, -(-int(c.lens[b]) // bs))] = -1 if b % 2 else c.kc.shape[0] + 5
    got = c.call(sv, handle)
    c.check(got)
    sv.specv_destroy(handle)


def test_attention_refuses_sequences(sv, h):
    """Bad lengths, parents and blocks: output 0, lse -inf and the bits, the
    other sequences as ever."""
    lens = [50, 3, 50, 50, 50, -1, 0, 33, 50]
    c = Case(8, "bf16", 9, 4, 4, 2, 64, 16, lens, "tree", width=4)
    c.lens[1] = 3  # below the rows
    c.lens[2] = 65  # past the table
    c.parents[3, 1] = 1  # itself
    c.parents[4, 0] = -2
    c.tables[7, 0] = c.kc.shape[0]  # outside the pool
    c.tables[8, 2] = -1
    got = c.call(sv, h)
    c.check(got)
    assert got["row_status"].tolist() == [0, 2048, 2048, 512, 512, 2048, 0, 4096, 4096]


def test_attention_takes_slices(sv, h):
    """Queries out of a fused projection, pools out of one tensor."""
    import torch

    c = Case(9, "bf16", 3, 5, 4, 2, 64, 16, [60, 5, 31], "tree")
    fused = torch.full((3, 5, 8, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    fused[:, :, 2:6] = c.q_t
    both = torch.full((c.kc_t.shape[0], 3, 2, 16, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    both[:, 0], both[:, 2] = c.kc_t, c.vc_t
    c.kc_t, c.vc_t = both[:, 0], both[:, 2]
    c.check(c.call(sv, h, q=fused[:, :, 2:6]))


@pytest.mark.parametrize("rows,hq", [(17, 8), (32, 16), (3, 8)])
def test_attention_of_one_query_for_all_rows(sv, h, rows, hq):
    """Queries that are one row expanded: a stride of zero."""
    c = Case(12, "bf16", 3, rows, hq, 2, 64, 16, [60, rows, 131], "tree")
    one = c.q_t[:1, :1].clone()
    c.q = np.broadcast_to(c.q[:1, :1], c.q.shape).copy()
    c.check(c.call(sv, h, q=one.expand(3, rows, hq, 64)))


@pytest.mark.parametrize("rows", [3, 20])
def test_attention_past_32_bit_offsets(sv, h, rows):
    """Blocks whose elements lie past 2^31."""
    import torch

    hkv, bs, dim = 8, 64, 128
    blocks = 2 ** 31 // (hkv * bs * dim) + 600
    c = Case(10, "bf16", 2, rows, 8, hkv, dim, bs, [200, 70], "tree")
    kc = torch.empty((blocks, hkv, bs, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty((blocks, hkv, bs, dim), dtype=torch.bfloat16, device="cuda")
    far = blocks - c.kc_t.shape[0]
    kc[far:], vc[far:] = c.kc_t, c.vc_t
    tables = np.where(c.tables >= 0, c.tables + far, -1).astype(np.int32)
    got = sv.specv_tree_attention(h, c.q_t, kc, vc, _dev(tables), _dev(c.lens), parents=_dev(c.parents), lse=True)
    torch.cuda.synchronize()
    c.check(got)


def test_attention_is_the_same_every_time(sv, h):
    import torch

    c = Case(11, "bf16", 5, 17, 8, 2, 128, 16, [3000, 17, 64, 1000, 0], "tree")
    one = c.call(sv, h)
    for _ in range(3):
        two = c.call(sv, h)
        for key in ("out", "lse"):
            assert torch.equal(one[key], two[key])


@pytest.mark.parametrize("rows", [1, 17, 32])
def test_attention_in_a_captured_graph(sv, h, rows):
    """Two graphs of the call, replayed with new lengths, tables and values."""
    import torch

    cases = [Case(20 + i, "bf16", 3, rows, 8, 2, 128, 16, lens, "tree", width=70)
             for i, lens in enumerate(([rows, 900, 100], [1000, rows + 1, 0]))]
    blocks = max(c.kc_t.shape[0] for c in cases)
    kc = torch.zeros((blocks, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    vc, q = torch.zeros_like(kc), torch.zeros_like(cases[0].q_t)
    tables = torch.zeros((3, 70), dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    par = torch.zeros((3, rows - 1), dtype=torch.int32, device="cuda")

    def call():
        return sv.specv_tree_attention(h, q, kc, vc, tables, lens, parents=par, lse=True)

    call()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(call())
    for c in cases + cases[::-1]:
        n = c.kc_t.shape[0]
        kc[:n], vc[:n] = c.kc_t, c.vc_t
        q.copy_(c.q_t)
        tables.copy_(_dev(c.tables))
        lens.copy_(_dev(c.lens))
        if rows > 1:
            par.copy_(_dev(c.parents))
        for g, out in zip(graphs, outs):
            out["out"].fill_(math.nan)
            g.replay()
            torch.cuda.synchronize()
            c.check(out)


def test_calls_on_two_streams(sv, h):
    """Calls in flight together on two streams keep apart."""
    import torch

    cases = [Case(30 + i, "bf16", 4, r, 8, 2, 128, 16, [5000, 40, 900, 2000], "tree")
             for i, r in enumerate((17, 5))]
    args = [(c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), _dev(c.parents)) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(6):
        for s, (q, k, v, t, n, p) in zip(streams, args):
            outs.append(sv.specv_tree_attention(h, q, k, v, t, n, parents=p, lse=True, stream=s))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        cases[i % 2].check(out)


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("use", [0, 3])
@pytest.mark.parametrize("rows,hq", [(17, 8), (32, 16)])
def test_withheld_copy_times_out_then_next_call_is_clean(sv, bs, use, rows, hq):
    """A slot of the tcgen05 kernel's first CTA is never filled: its waits run
    out, the sequences it works on report bit 64, the others and the next
    call are as ever.  (370 tiles and more for 152 CTAs: a run is two tiles at
    least, four slot uses.)"""
    import torch

    handle = sv.specv_create(0, max_batch=64, max_k=31, vocab=1000)
    c = Case(50 + use, "bf16", 4, rows, hq, 2, 128, bs, [5900, 6000, 6200, 6100], "tree")
    sv.specv_test_withhold_stage(handle, use, 200_000)
    got = c.call(sv, handle)
    again = c.call(sv, handle)
    c.check(again)
    late = (got["row_status"] & sv.ST_TIMEOUT) != 0
    assert late[0] and late.sum() < 4 and not (got["row_status"] & ~sv.ST_TIMEOUT).any()
    for key in ("out", "lse"):
        assert torch.equal(got[key][~late], again[key][~late])
    sv.specv_destroy(handle)


def test_many_calls_give_the_same(sv, h):
    """Many calls back to back under memory load, every one the same bits
    (a slot read too early would show)."""
    import torch

    c = Case(60, "bf16", 24, 17, 8, 2, 128, 16, [700 + 97 * (i % 9) for i in range(24)], "tree")
    args = (c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens))
    par = _dev(c.parents)
    one = sv.specv_tree_attention(h, *args, parents=par, lse=True)
    c.check(one)
    noise = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(300):
        if i % 10 == 0:
            with torch.cuda.stream(side):
                noise.add_(1)
        two = sv.specv_tree_attention(h, *args, parents=par, lse=True)
        wrong += (two["out"] != one["out"]).sum() + (two["lse"] != one["lse"]).sum()
    torch.cuda.synchronize()
    assert int(wrong) == 0


# ---------------------------------------------------------------------------- append
APPENDS = [
    # B, rows, q heads, kv heads, dim, block, lengths, tree, rot, interleaved, counts
    (1, 1, 4, 1, 64, 16, [1], "chain", 64, False, None),
    (3, 1, 8, 2, 128, 16, [1, 0, 999], "chain", 128, False, None),
    (3, 6, 6, 3, 80, 5, [6, 7, 40], "chain", 40, True, None),
    (2, 17, 8, 2, 128, 16, [17, 300], "tree", 128, False, None),
    (2, 32, 4, 4, 64, 7, [64, 33], "star", 32, True, None),
    (2, 12, 2, 1, 256, 16, [100, 12], "tree", 256, True, None),
    (3, 100, 4, 2, 64, 16, [100, 120, 43], "chain", 64, False, [100, 37, 0]),
    (3, 5, 4, 2, 16, 1, [5, 4, 9], "tree", 6, False, [5, 2, 3]),
    (2, 4, 2, 1, 48, 16, [130000, 5], "chain", 48, False, None),
    (2, 3, 2, 2, 96, 16, [20, 4], "tree", 0, False, None),
    (2, 300, 3, 1, 32, 64, [700, 300], "chain", 30, True, None),
]


def _append_case(seed, dtype, B, rows, hq, hkv, dim, bs, lens, kind, rot):
    rng = np.random.default_rng(seed)
    lens = np.array(lens, np.int32)
    tables, blocks = _tables(rng, np.maximum(lens, 0), bs)
    pools = [_rounded(rng, (blocks, hkv, bs, dim), dtype) for _ in range(2)]
    rows_ = [_rounded(rng, (B, rows, n, dim), dtype) for n in (hq, hkv, hkv)]
    inv = None if rot == 0 else (10000.0 ** (-np.arange(rot // 2) * 2 / rot)).astype(np.float32)
    return rng, lens, tables, pools, rows_, inv, _random_tree(rng, kind, B, rows)


def _append_bound(got, ref, x0, x1, half):
    """Each output is x0 c - x1 s in fp32: c and s are off by 2^-22 (the angle
    in fp32 within [-pi, pi], 2^-23, and sincosf's 2 ulp), the products and
    the sum round once each (2^-24 of |x0| + |x1| apiece), and the result once
    to its type."""
    mag = np.abs(x0) + np.abs(x1)
    assert (np.abs(got - ref) <= half * np.abs(ref) + 2.0 ** -21 * mag).all(), np.max(np.abs(got - ref))


def _partner(x, rot, inter):
    """The other value of each value's pair (0 outside the rotated part)."""
    y = np.zeros_like(x)
    if rot:
        if inter:
            y[..., 0:rot:2], y[..., 1:rot:2] = x[..., 1:rot:2], x[..., 0:rot:2]
        else:
            y[..., :rot // 2], y[..., rot // 2:rot] = x[..., rot // 2:rot], x[..., :rot // 2]
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", APPENDS, ids=lambda s: "B%d_R%d_H%d-%d_D%d_bs%d_%s" % (s[:6] + (s[7],)))
def test_append_matches_the_formula(sv, h, dtype, shape):
    import torch

    B, rows, hq, hkv, dim, bs, lens, kind, rot, inter, counts = shape
    half = BF16_HALF if dtype == "bf16" else F32_HALF
    rng, lens, tables, pools, xs, inv, par = _append_case(rows, _dtype(dtype), B, rows, hq, hkv, dim, bs, lens, kind, rot)
    (kc_t, kc), (vc_t, vc) = pools
    (q_t, q), (k_t, k), (v_t, v) = xs
    counts = None if counts is None else np.array(counts, np.int32)
    before = _np(kc_t)
    got = sv.specv_cache_append(h, kc_t, vc_t, _dev(tables), _dev(lens), k_t, v_t, q=q_t,
                                inv_freq=None if inv is None else _dev(inv), interleaved=inter,
                                parents=None if par is None else _dev(par),
                                row_counts=None if counts is None else _dev(counts))
    torch.cuda.synchronize()
    ref_k, ref_v = kc.copy(), vc.copy()
    q_out, status, written = P.append(ref_k, ref_v, tables, lens, k, v, q=q, inv_freq=inv, interleaved=inter,
                                      parents=par, counts=counts)
    np.testing.assert_array_equal(got["row_status"].cpu().numpy(), status)
    np.testing.assert_array_equal(_np(vc_t), ref_v)  # values are moved, bit by bit
    kg = _np(kc_t)
    hit = np.zeros((kc.shape[0], bs), bool)
    for blk, slot in written:
        hit[blk, slot] = True
    rest = ~np.broadcast_to(hit[:, None, :, None], kc.shape)
    np.testing.assert_array_equal(kg[rest], before[rest])  # nothing else is touched
    peer = kc.copy()
    P.append(peer, vc.copy(), tables, lens, _partner(k, rot, inter), v, counts=counts, parents=par)
    own = kc.copy()
    P.append(own, vc.copy(), tables, lens, k, v, counts=counts, parents=par)
    _append_bound(kg[~rest], ref_k[~rest], own[~rest], peer[~rest], half)
    _append_bound(_np(got["q_out"]), q_out, q, _partner(q, rot, inter), half)
    for b in range(B):
        m = rows if counts is None else counts[b]
        if lens[b] == 0 or status[b]:
            m = 0
        assert np.all(_np(got["q_out"])[b, m:] == 0)


# more tokens than the SMs hold at once: CTAs of fewer threads
MANY_APPENDS = [
    (60, 17, 4, 2, 64, 16, [17 + i if i % 7 else 0 for i in range(60)], "tree", 64, False, None),
    (3, 300, 6, 3, 80, 5, [300, 417, 299], "chain", 40, True, [300, 291, 0]),
    (300, 3, 2, 1, 16, 1, [3 + i % 5 for i in range(300)], "tree", 6, False, [i % 4 for i in range(300)]),
    (100, 9, 2, 1, 256, 16, [9 + i for i in range(100)], "star", 256, False, None),
    (1, 777, 8, 4, 48, 64, [1000], "chain", 0, False, [770]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", MANY_APPENDS, ids=lambda s: "B%d_R%d_H%d-%d_D%d_bs%d_%s" % (s[:6] + (s[7],)))
def test_append_of_many_tokens(sv, h, dtype, shape):
    test_append_matches_the_formula(sv, h, dtype, shape)


def test_append_without_queries_in_place_and_in_slices(sv, h):
    import torch

    rng, lens, tables, pools, xs, inv, par = _append_case(3, torch.bfloat16, 2, 5, 4, 2, 64, 16, [30, 5], "tree", 64)
    (kc, _), (vc, _) = pools
    (q, _), (k, _), (v, _) = xs
    args = dict(inv_freq=_dev(inv), parents=_dev(par))
    fused = torch.zeros((2, 5, 9, 64), dtype=torch.bfloat16, device="cuda")
    fused[:, :, :4], fused[:, :, 4:6], fused[:, :, 6:8] = q, k, v
    k1, v1, k2, v2 = kc.clone(), vc.clone(), kc.clone(), vc.clone()
    one = sv.specv_cache_append(h, k1, v1, _dev(tables), _dev(lens), k, v, q=q, **args)
    none = sv.specv_cache_append(h, k2, v2, _dev(tables), _dev(lens), fused[:, :, 4:6], fused[:, :, 6:8], **args)
    assert "q_out" not in none and torch.equal(k1, k2) and torch.equal(v1, v2)
    two = sv.specv_cache_append(h, k2, v2, _dev(tables), _dev(lens), k, v, q=fused[:, :, :4], **args)
    assert torch.equal(one["q_out"], two["q_out"])
    qq = q.clone()
    sv.specv_cache_append(h, k2, v2, _dev(tables), _dev(lens), k, v, q=qq, out={"q_out": qq}, **args)
    assert torch.equal(qq, one["q_out"]) and torch.equal(k1, k2)


def test_append_refuses_sequences(sv, h):
    """Nothing of a refused sequence is written; the others are."""
    import torch

    B, rows = 8, 4
    lens = [20, 3, 65, 20, 20, -4, 40, 20]
    rng, lens, tables, pools, xs, inv, par = _append_case(4, torch.float32, B, rows, 2, 2, 32, 16,
                                                          [20, 20, 64, 20, 20, 0, 40, 20], "tree", 32)
    lens = np.array([20, 3, 65, 20, 20, -4, 40, 20], np.int32)
    par[3, 2] = 2
    par[4, 0] = -9
    tables[6, 2] = -1  # the block of the rows
    tables[7, 0] = 10 ** 6  # a block before them
    (kc_t, kc), (vc_t, vc) = pools
    (q_t, q), (k_t, k), (v_t, v) = xs
    got = sv.specv_cache_append(h, kc_t, vc_t, _dev(tables), _dev(lens), k_t, v_t, q=q_t, inv_freq=_dev(inv),
                                parents=_dev(par))
    torch.cuda.synchronize()
    status = got["row_status"].tolist()
    assert status == [0, 2048, 2048, 512, 512, 2048, 4096, 0]
    P.append(kc, vc, tables, lens, k, v, q=q, inv_freq=inv, parents=par)
    np.testing.assert_array_equal(_np(vc_t), vc)
    assert np.max(np.abs(_np(kc_t) - kc)) < 2.0 ** -19
    bad = np.array(status) != 0
    assert np.all(_np(got["q_out"])[bad] == 0) and np.all(_np(got["q_out"])[~bad].any((1, 2, 3)))
    counts = np.array([4, 5, 0, -1, 4, 0, 1, 2], np.int32)
    got = sv.specv_cache_append(h, kc_t, vc_t, _dev(tables), _dev(np.full(8, 20, np.int32)), k_t, v_t,
                                row_counts=_dev(counts))
    assert got["row_status"].tolist() == [0, 2048, 0, 2048, 0, 0, 0, 0]


def test_append_far_positions(sv, h):
    """Angles far out: position 2^30 in a table of large blocks."""
    import torch

    rng = np.random.default_rng(2)
    bs, n = 65536, 2 ** 30 + 3
    tables = np.full((1, n // bs + 1), -1, np.int32)
    tables[0, -1] = 1
    kc = torch.zeros((2, 1, bs, 16), device="cuda")
    vc = torch.zeros_like(kc)
    k_t, k = _rounded(rng, (1, 2, 1, 16), torch.float32)
    inv = np.array([1.0, 0.333, 0.01, 1e-4, 0.77, 1e-6, 0.5, 3.0], np.float32)
    sv.specv_cache_append(h, kc, vc, _dev(tables), _dev(np.array([n], np.int32)), k_t, k_t, inv_freq=_dev(inv))
    torch.cuda.synchronize()
    for r in range(2):
        ref = P.rotate(k[0, r], n - 2 + r, inv, False)
        _append_bound(_np(kc[1, :, (n - 2 + r) % bs]), ref, k[0, r], _partner(k[0, r], 16, False), F32_HALF)


# ---------------------------------------------------------------------------- compaction
def _paths(rng, B, M):
    path, kept = np.full((B, M), -1, np.int32), rng.integers(0, M + 1, size=B).astype(np.int32)
    kept[0] = M
    for b in range(B):
        path[b, :kept[b]] = np.sort(rng.permutation(M)[:kept[b]])
    return path, kept


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,M,layers,hkv,dim,bs,lens", [(1, 1, 1, 1, 16, 1, [1]), (3, 6, 1, 2, 64, 5, [6, 0, 50]),
                                                       (5, 31, 3, 4, 128, 16, [31, 40, 64, 100, 33]),
                                                       (4, 17, 7, 3, 80, 16, [20, 17, 35, 200])])
def test_compaction_matches(sv, h, dtype, B, M, layers, hkv, dim, bs, lens):
    import torch

    rng = np.random.default_rng(B + M)
    lens = np.array(lens, np.int32)
    tables, blocks = _tables(rng, lens, bs)
    (kc_t, kc), (vc_t, vc) = [_rounded(rng, (layers, blocks, hkv, bs, dim), _dtype(dtype)) for _ in range(2)]
    path, kept = _paths(rng, B, M)
    st = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    sv.specv_cache_compact(h, kc_t, vc_t, _dev(tables), _dev(lens), _dev(path), _dev(kept), row_status=st)
    torch.cuda.synchronize()
    status = P.compact(kc, vc, tables, lens, path, kept)
    assert st.tolist() == status.tolist() == [0] * B
    np.testing.assert_array_equal(_np(kc_t), kc)
    np.testing.assert_array_equal(_np(vc_t), vc)


def test_compaction_of_interleaved_layers(sv, h):
    """[blocks, layers, ...] pools: the layers' stride below the blocks'."""
    import torch

    rng = np.random.default_rng(12)
    lens = np.array([20, 9], np.int32)
    tables, blocks = _tables(rng, lens, 4)
    (k_t, k), (v_t, v) = [_rounded(rng, (blocks, 3, 2, 4, 16), torch.bfloat16) for _ in range(2)]
    path, kept = _paths(rng, 2, 8)
    sv.specv_cache_compact(h, k_t.transpose(0, 1), v_t.transpose(0, 1), _dev(tables), _dev(lens), _dev(path),
                           _dev(kept))
    torch.cuda.synchronize()
    P.compact(k.transpose(1, 0, 2, 3, 4), v.transpose(1, 0, 2, 3, 4), tables, lens, path, kept)
    np.testing.assert_array_equal(_np(k_t), k)
    np.testing.assert_array_equal(_np(v_t), v)


def test_compaction_refuses_sequences(sv, h):
    import torch

    rng = np.random.default_rng(13)
    M, bs = 5, 4
    lens = np.array([10, 4, 21, 10, 10, 10, 10, 10, 0], np.int32)
    tables, blocks = _tables(rng, np.where(lens == 21, 20, lens), bs)
    path = np.tile(np.array([0, 2, 3, -1, -1], np.int32), (9, 1))
    kept = np.full(9, 3, np.int32)
    kept[3], kept[4] = 6, -1
    path[5] = [2, 2, 3, -1, -1]
    path[6] = [1, 4, 5, -1, -1]
    tables[7, 2] = blocks
    (kc_t, kc), (vc_t, vc) = [_rounded(rng, (2, blocks, 1, bs, 16), torch.float32) for _ in range(2)]
    st = torch.full((9,), -7, dtype=torch.int32, device="cuda")
    sv.specv_cache_compact(h, kc_t, vc_t, _dev(tables), _dev(lens), _dev(path), _dev(kept), row_status=st)
    torch.cuda.synchronize()
    status = P.compact(kc, vc, tables, lens, path, kept)
    assert st.tolist() == status.tolist() == [0, 2048, 2048, 128, 128, 8192, 8192, 4096, 0]
    np.testing.assert_array_equal(_np(kc_t), kc)
    np.testing.assert_array_equal(_np(vc_t), vc)


# ---------------------------------------------------------------------------- refusals of the call
def test_calls_are_refused_without_launching(sv, h):
    import torch

    c = Case(40, "bf16", 2, 3, 4, 2, 64, 16, [20, 9], "tree")
    t, n, p = _dev(c.tables), _dev(c.lens), _dev(c.parents)
    before = sv.specv_launch_count(h)

    def attn(**kw):
        a = dict(q=c.q_t, k=c.kc_t, v=c.vc_t, t=t, n=n, parents=p)
        a.update(kw)
        return sv.specv_tree_attention(h, a.pop("q"), a.pop("k"), a.pop("v"), a.pop("t"), a.pop("n"), **a)

    for exc, kw in [(TypeError, dict(q=c.q_t.float())), (ValueError, dict(q=c.q_t[:1])),
                    (ValueError, dict(q=c.q_t[:, :, :, :32])), (TypeError, dict(v=c.vc_t.float())),
                    (ValueError, dict(v=c.vc_t[1:])), (ValueError, dict(k=c.kc_t.transpose(1, 2))),
                    (ValueError, dict(n=n[:1])), (TypeError, dict(n=n.long())), (ValueError, dict(parents=p[:, :1])),
                    (TypeError, dict(t=c.tables)), (sv.SpecvError, dict(scale=math.nan)),
                    (sv.SpecvError, dict(q=c.q_t[:, :, :3], parents=p)),
                    (ValueError, dict(q=c.q_t.expand(2, 3, 4, 64)[:, :, ::2]))]:
        with pytest.raises(exc):
            attn(**kw)
    wide = torch.zeros((2, 33, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(sv.SpecvError):
        attn(q=wide, parents=None)  # more rows than max_k + 1
    odd = torch.zeros((3, 2, 16, 24), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(sv.SpecvError):
        attn(q=torch.zeros((2, 3, 4, 24), dtype=torch.bfloat16, device="cuda"), k=odd, v=odd)  # head_dim 24
    need = sv.specv_tree_attention_workspace(h, sv.SPECV_BF16, 2, 64, 4, 2, 3)
    if need:
        with pytest.raises(sv.SpecvError):
            attn(workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    kv = c.kc_t[:2].reshape(2, 2, 2, 8, 64)
    rows = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16, device="cuda")
    inv = torch.ones(33, device="cuda")
    with pytest.raises(sv.SpecvError):
        sv.specv_cache_append(h, c.kc_t, c.vc_t, t, n, rows, rows, inv_freq=inv)  # 66 rotated values of 64
    with pytest.raises(ValueError):
        sv.specv_cache_append(h, c.kc_t, c.vc_t, t, n, rows, rows[:, :2])
    with pytest.raises(ValueError):
        sv.specv_cache_append(h, kv, kv, t, n, rows, rows)
    with pytest.raises(ValueError):
        sv.specv_cache_compact(h, c.kc_t, c.vc_t, t, n, p, n[:1])
    with pytest.raises(sv.SpecvError):
        sv.specv_cache_compact(h, c.kc_t, c.vc_t, t, n, torch.zeros((2, 32), dtype=torch.int32, device="cuda"), n)
    assert sv.specv_launch_count(h) == before


def test_attention_is_refused_in_place(sv, h):
    """out that is q itself: rows would be written while others read theirs."""
    c = Case(41, "bf16", 2, 3, 4, 2, 64, 16, [20, 9], "tree")
    before = sv.specv_launch_count(h)
    with pytest.raises(sv.SpecvError):
        sv.specv_tree_attention(h, c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), out=dict(out=c.q_t))
    assert sv.specv_launch_count(h) == before


def test_empty_batches_and_empty_pools(sv, h):
    import torch

    z = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    i = torch.int32
    pool = z(3, 2, 16, 64)
    before = sv.specv_launch_count(h)
    sv.specv_tree_attention(h, z(0, 2, 4, 64), pool, pool, z(0, 4, d=i), z(0, d=i))
    sv.specv_cache_append(h, pool, pool, z(0, 4, d=i), z(0, d=i), z(0, 2, 2, 64), z(0, 2, 2, 64))
    sv.specv_cache_compact(h, pool, pool, z(0, 4, d=i), z(0, d=i), z(0, 3, d=i), z(0, d=i))
    assert sv.specv_launch_count(h) == before
    none = z(0, 2, 16, 64)
    got = sv.specv_tree_attention(h, z(2, 2, 4, 64) + 1, none, none, z(2, 0, d=i), z(2, d=i), lse=True)
    assert got["row_status"].tolist() == [0, 0] and not got["out"].any() and torch.isneginf(got["lse"]).all()
    many = torch.full((2,), 20, dtype=i, device="cuda")
    got = sv.specv_tree_attention(h, z(2, 20, 4, 64) + 1, none, none, z(2, 2, d=i), many, lse=True)
    assert got["row_status"].tolist() == [4096, 4096] and not got["out"].any()
    one = torch.ones(2, dtype=i, device="cuda")
    got = sv.specv_tree_attention(h, z(2, 1, 4, 64) + 1, none, none, z(2, 1, d=i), one, lse=True)
    assert got["row_status"].tolist() == [4096, 4096] and not got["out"].any()
    got = sv.specv_cache_append(h, none, none, z(2, 1, d=i), one, z(2, 1, 2, 64), z(2, 1, 2, 64))
    assert got["row_status"].tolist() == [4096, 4096]


def test_layers_of_zero_and_paths_of_one(sv, h):
    import torch

    i = torch.int32
    pool = torch.zeros((1, 4, 2, 16, 16), dtype=torch.bfloat16, device="cuda")
    lens, table = _dev(np.array([9, 3], np.int32)), _dev(np.array([[1], [0]], np.int32))
    path, acc = _dev(np.array([[0], [5]], np.int32)), _dev(np.array([1, 1], np.int32))
    st = torch.full((2,), -7, dtype=i, device="cuda")
    sv.specv_cache_compact(h, pool, pool, table, lens, path, acc, row_status=st)
    assert st.tolist() == [0, 8192]
    with pytest.raises(sv.SpecvError):
        sv.specv_cache_compact(h, pool[:0], pool[:0], table, lens, path, acc)


def test_calls_in_one_captured_graph(sv):
    """Append, attention and compaction in a graph, replayed as the sequences
    grow: the same as eager calls."""
    import torch

    B, M, hq, hkv, dim, bs = 3, 6, 8, 2, 64, 16
    rng = np.random.default_rng(3)
    h1 = sv.specv_create(0, max_batch=B, max_k=M, vocab=50)
    inv = _dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
    tables = _dev(rng.permutation(3 * 8).reshape(3, 8).astype(np.int32))
    par = _dev(_random_tree(rng, "tree", B, M + 1))
    path, acc = _dev(np.array([[1, 3, 5, -1, -1, -1]] * B, np.int32)), _dev(np.array([3, 0, 2], np.int32))

    def state():
        g = torch.Generator(device="cuda").manual_seed(5)
        pool = torch.randn((2, 24, hkv, bs, dim), generator=g, device="cuda").to(torch.bfloat16)
        return dict(k=pool[0].clone(), v=pool[1].clone(), lens=_dev(np.array([20, 7, 50], np.int32)),
                    x=torch.zeros((B, M + 1, hq + 2 * hkv, dim), dtype=torch.bfloat16, device="cuda"))

    def step(s):
        x = s["x"]
        rot = sv.specv_cache_append(h1, s["k"], s["v"], tables, s["lens"], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:],
                                    q=x[:, :, :hq], inv_freq=inv, parents=par)
        got = sv.specv_tree_attention(h1, rot["q_out"], s["k"], s["v"], tables, s["lens"], parents=par, lse=True)
        sv.specv_cache_compact(h1, s["k"], s["v"], tables, s["lens"], path, acc)
        return rot["q_out"], got["out"], got["lse"]

    eager, captured = state(), state()
    step(captured)
    torch.cuda.synchronize()
    fresh = state()
    for key in captured:
        captured[key].copy_(fresh[key])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(captured)
    for i in range(4):
        x = torch.randn(eager["x"].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))
        for s in (eager, captured):
            s["x"].copy_(x)
            s["lens"].add_(3 * i)
        want = step(eager)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
        assert torch.equal(eager["k"], captured["k"]) and torch.equal(eager["v"], captured["v"])
    sv.specv_destroy(h1)


# ---------------------------------------------------------------------------- together
def test_a_verify_round_of_all_of_them(sv):
    """Rounds of append, tree attention, greedy tree verification, compaction
    and rollback against a dense history: after each round the cache holds
    the accepted tokens' rotated keys and their values, in order, and the
    next round attends to exactly these."""
    import torch

    B, M, hq, hkv, dim, bs, V, layers = 4, 9, 4, 2, 64, 4, 50, 3
    rng = np.random.default_rng(77)
    hv = sv.specv_create(0, max_batch=B, max_k=M, vocab=V)
    inv = (10000.0 ** (-np.arange(dim // 2) * 2 / dim)).astype(np.float32)
    max_blocks = 30
    kc = torch.zeros((layers, B * max_blocks, hkv, bs, dim), dtype=torch.float32, device="cuda")
    vc = torch.zeros_like(kc)
    tables = torch.full((B, max_blocks), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    blocks = torch.zeros(B, dtype=torch.int32, device="cuda")
    free = [int(x) for x in rng.permutation(B * max_blocks)]
    free_list = torch.zeros(B * max_blocks, dtype=torch.int32, device="cuda")
    free_count = torch.zeros(1, dtype=torch.int32, device="cuda")
    hist_k = [[np.zeros((0, hkv, dim)) for _ in range(B)] for _ in range(layers)]
    hist_v = [[np.zeros((0, hkv, dim)) for _ in range(B)] for _ in range(layers)]

    def reserve(counts):
        nb, ln, tb = blocks.tolist(), lens.tolist(), tables.cpu().numpy()
        for b in range(B):
            ln[b] += counts[b]
            while nb[b] * bs < ln[b]:
                tb[b, nb[b]] = free.pop()
                nb[b] += 1
        tables.copy_(_dev(tb))
        blocks.copy_(_dev(np.array(nb, np.int32)))
        lens.copy_(_dev(np.array(ln, np.int32)))

    def check_history():
        for l in range(layers):
            for b in range(B):
                n = int(lens[b])
                assert n == len(hist_k[l][b])
                t = np.arange(n)
                ids = tables[b].cpu().numpy()[t // bs]
                assert np.max(np.abs(_np(kc[l])[ids, :, t % bs] - hist_k[l][b]), initial=0) < 2.0 ** -18
                np.testing.assert_array_equal(_np(vc[l])[ids, :, t % bs], hist_v[l][b])

    # prompts, padded to the longest
    counts = np.array([13, 1, 7, 0], np.int32)
    reserve(counts.tolist())
    for l in range(layers):
        (k_t, k), (v_t, v) = [_rounded(rng, (B, 13, hkv, dim), torch.float32) for _ in range(2)]
        sv.specv_cache_append(hv, kc[l], vc[l], tables, lens, k_t, v_t, inv_freq=_dev(inv), row_counts=_dev(counts))
        for b in range(B):
            hist_k[l][b] = np.array([P.rotate(k[b, r], r, inv, False) for r in range(counts[b])]).reshape(-1, hkv, dim)
            hist_v[l][b] = v[b, :counts[b]]
    check_history()
    for step in range(5):
        parents = _random_tree(rng, "tree", B, M + 1)
        par_t = _dev(parents)
        reserve([M + 1] * B)
        new = []
        for l in range(layers):
            (q_t, q), (k_t, k), (v_t, v) = [_rounded(rng, (B, M + 1, n, dim), torch.float32) for n in (hq, hkv, hkv)]
            rot = sv.specv_cache_append(hv, kc[l], vc[l], tables, lens, k_t, v_t, q=q_t, inv_freq=_dev(inv),
                                        parents=par_t)
            got = sv.specv_tree_attention(hv, rot["q_out"], kc[l], vc[l], tables, lens, parents=par_t, lse=True)
            kk, vv = np.zeros((B, M + 1, hkv, dim)), v
            for b in range(B):
                _, depth, seen = P.tree(parents[b], M + 1)
                n = len(hist_k[l][b])
                for r in range(M + 1):
                    kk[b, r] = P.rotate(k[b, r], n + depth[r], inv, False)
                for r in range(M + 1):
                    qq = P.rotate(q[b, r], n + depth[r], inv, False)
                    K = np.concatenate([hist_k[l][b], kk[b, sorted(seen[r])]])
                    W = np.concatenate([hist_v[l][b], vv[b, sorted(seen[r])]])
                    for hh in range(hq):
                        s = K[:, hh // 2] @ qq[hh] * dim ** -0.5
                        e = np.exp(s - s.max())
                        o = e @ W[:, hh // 2] / e.sum()
                        # fp32 throughout: scores off by 2^-23 * (dim + 16) * ~20 at most, as in attention_bounds
                        assert np.max(np.abs(_np(got["out"][b, r, hh]) - o)) < 2e-3 * np.abs(W).max()
            new.append((kk, vv))
        tokens = rng.integers(0, V, size=(B, M)).astype(np.int32)
        logits = rng.normal(size=(B, M + 1, V)).astype(np.float32)
        for b in range(B):  # most nodes are what their parent's row predicts
            for i in range(M):
                if rng.random() < 0.8:
                    logits[b, parents[b, i] + 1, tokens[b, i]] = 9.0 + i
        ver = sv.specv_verify_tree_greedy(hv, _dev(logits), _dev(tokens), par_t)
        st = torch.empty(B, dtype=torch.int32, device="cuda")
        sv.specv_cache_compact(hv, kc, vc, tables, lens, ver["path"], ver["num_accepted"], row_status=st)
        assert st.tolist() == [0] * B
        free_count.zero_()
        sv.specv_rollback(hv, ver["num_accepted"], M, lens, tables, blocks, bs, free_list, free_count)
        torch.cuda.synchronize()
        free.extend(free_list[:int(free_count)].tolist())
        path, acc = ver["path"].cpu().numpy(), ver["num_accepted"].tolist()
        assert max(acc) > 1
        for l in range(layers):
            for b in range(B):
                rows = [0] + [1 + int(x) for x in path[b, :acc[b]]]
                hist_k[l][b] = np.concatenate([hist_k[l][b], new[l][0][b, rows]])
                hist_v[l][b] = np.concatenate([hist_v[l][b], new[l][1][b, rows]])
        check_history()
    sv.specv_destroy(hv)
