"""GPU parity of attention over a shared prefix with its plain float64
restatement (serving_plain.py)."""
import math

import numpy as np
import pytest

import cache_plain as P
import serving_plain as S
from test_gpu_cache import _dev, _dtype, _np, _random_tree, _rounded, h, sv  # noqa: F401

pytestmark = pytest.mark.gpu


class Shared:
    """Inputs of a call: lens are the sequences' own positions behind the prefix (0: idle); positions that nobody holds
    are NaN, and the sequences' own tables name nothing of the prefix."""

    def __init__(self, seed, dtype, B, rows, hq, hkv, dim, bs, prefix, lens, kind="tree", q_scale=1.5):
        import torch

        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.rows, self.prefix, self.bs = rng, _dtype(dtype), rows, prefix, bs
        assert len(lens) == B and prefix % bs == 0
        self.lens = np.array([n + prefix if n > 0 else n for n in lens], np.int32)
        n0 = prefix // bs
        used = [-(-max(int(n), 0) // bs) for n in lens]
        order = rng.permutation(n0 + sum(used) + 3)
        self.table0 = np.array(order[:n0], np.int32)
        self.tables = np.full((B, n0 + max(used + [1])), -7, np.int32)
        at = n0
        for b, n in enumerate(used):
            self.tables[b, n0:n0 + n] = order[at:at + n]
            at += n
        blocks = len(order)
        self.kc_t, _ = _rounded(rng, (blocks, hkv, bs, dim), self.dtype)
        self.vc_t, _ = _rounded(rng, (blocks, hkv, bs, dim), self.dtype)
        held = np.zeros((blocks, bs), bool)
        held[self.table0] = True
        for b, n in enumerate(lens):
            t = np.arange(max(int(n), 0))
            held[self.tables[b, n0 + t // bs], t % bs] = True
        hole = torch.from_numpy(~held).cuda()[:, None, :, None]
        self.kc_t.masked_fill_(hole, math.nan)
        self.vc_t.masked_fill_(hole, math.nan)
        self.q_t, self.q = _rounded(rng, (B, rows, hq, dim), self.dtype, q_scale)
        self.parents = _random_tree(rng, kind, B, rows)
        self.scale = dim ** -0.5
        self.ref = None

    def args(self):
        return (self.q_t, self.kc_t, self.vc_t, _dev(self.tables), _dev(self.lens), _dev(self.table0),
                _dev(np.array([self.prefix], np.int32)))

    def call(self, sv, h, **kw):  # noqa: F811
        import torch

        par = None if self.parents is None else _dev(self.parents)
        got = sv.specv_prefix_attention(h, *self.args(), parents=par, lse=True, **kw)
        torch.cuda.synchronize()
        return got

    def check(self, got, scale=None):
        scale = self.scale if scale is None else scale
        if self.ref is None or self.ref[0] != scale:
            self.ref = scale, S.prefix_attention(self.q, _np(self.kc_t), _np(self.vc_t), self.tables, self.lens, self.table0,
                                                 self.prefix, self.parents, scale)
        out, lse, status, avg, mag = self.ref[1]
        np.testing.assert_array_equal(got["row_status"].cpu().numpy(), status)
        g, gl = _np(got["out"]), _np(got["lse"])
        np.testing.assert_array_equal(np.isnan(g), np.isnan(out))
        np.testing.assert_array_equal(g[np.isinf(out)], out[np.isinf(out)])
        fin = np.isfinite(lse)
        t_out, t_lse = P.attention_bounds(out, np.where(fin, lse, 0), avg, mag, int(self.lens[status == 0].max(initial=1)),
                                          self.q.shape[-1], str(self.dtype).endswith("bfloat16"))
        same = np.isfinite(out)
        bad = same & ~(np.abs(g - np.where(same, out, 0)) <= t_out)
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], g[bad][:4], out[bad][:4], t_out[bad][:4])
        np.testing.assert_array_equal(gl[~fin], lse[~fin])
        bad = fin & ~(np.abs(gl - np.where(fin, lse, 0)) <= t_lse)
        assert not bad.any(), (gl[bad][:4], lse[bad][:4], t_lse[bad][:4])


# B, rows, q heads, kv heads, dim, block, prefix, own positions, tree
SHAPES = [
    (1, 1, 1, 1, 16, 1, 1, [1], "chain"),
    (1, 1, 4, 2, 64, 16, 0, [5], "chain"),              # no prefix
    (3, 1, 8, 2, 128, 16, 16, [1, 0, 40], "chain"),
    (4, 1, 32, 8, 128, 16, 256, [1, 33, 64, 200], "chain"),
    (20, 1, 8, 2, 128, 16, 400, [1 + 7 * i for i in range(20)], "chain"),
    (5, 3, 6, 2, 80, 5, 135, [3, 0, 64, 65, 131], "tree"),
    (3, 17, 8, 2, 128, 16, 1024, [17, 30, 200], "tree"),   # prefix rows in two tiles, own in one
    (9, 17, 8, 2, 128, 16, 528, [17 + 20 * i if i != 4 else 0 for i in range(9)], "tree"),
    (3, 20, 6, 2, 48, 8, 128, [21, 128, 260], "tree"),
    (2, 24, 10, 2, 80, 64, 192, [24, 200], "star"),
    (4, 18, 14, 2, 112, 128, 256, [130, 270, 18, 19], "tree"),
    (3, 32, 16, 2, 128, 256, 512, [255, 600, 32], "tree"),
    (3, 32, 16, 2, 64, 24, 480, [96, 420, 0], "tree"),
    (2, 32, 24, 1, 64, 1, 131, [32, 135], "line"),
    (2, 9, 24, 1, 256, 16, 160, [9, 150], "tree"),
    (17, 1, 2, 2, 256, 8, 200, [1 + i for i in range(17)], "chain"),
    (3, 31, 5, 5, 48, 3, 300, [31, 95, 96], "tree"),
    (70, 2, 4, 4, 64, 16, 64, [2 + 3 * i for i in range(70)], "tree"),
    (300, 1, 4, 1, 128, 16, 320, [1 + i % 40 for i in range(300)], "chain"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "B%d_R%d_H%d-%d_D%d_bs%d_p%d" % s[:7])
def test_prefix_attention_matches_the_formula(sv, h, dtype, shape):  # noqa: F811
    c = Shared(sum(shape[:7]), dtype, *shape)
    c.check(c.call(sv, h))


@pytest.mark.parametrize("dtype,B,rows,hq,hkv,prefix", [("bf16", 4, 1, 8, 2, 20000), ("bf16", 2, 17, 8, 2, 9600),
                                                        ("bf16", 20, 5, 8, 1, 6400), ("f32", 3, 5, 4, 2, 9600)])
def test_prefix_attention_over_a_long_prefix(sv, h, dtype, B, rows, hq, hkv, prefix):  # noqa: F811
    c = Shared(prefix + rows, dtype, B, rows, hq, hkv, 128, 16, prefix, [rows + 37 * i for i in range(B)])
    c.check(c.call(sv, h))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,rows", [(6, 1), (6, 17)])
def test_prefix_attention_refuses_sequences(sv, h, dtype, B, rows):  # noqa: F811
    import torch

    c = Shared(3, dtype, B, rows, 8, 2, 64, 16, 160, [rows, 0, 50, 60, 70, 80])
    c.lens[2], c.lens[5] = 160 + rows - 1, -3
    c.tables[3, 11] = 10 ** 6
    if rows > 1:
        c.parents[4, 3] = 3
    c.check(c.call(sv, h))
    assert c.ref[1][2].tolist() == [0, 0, 2048, 4096, 512 if rows > 1 else 0, 2048]
    for low in (-2 ** 31, -2 ** 31 + 5, 2 ** 31 - 1):  # nothing is taken off a length that has too little
        lens, c.ref = c.lens.copy(), None
        c.lens[5], c.lens[0] = low, low
        c.check(c.call(sv, h))
        c.lens, c.ref = lens, None
    # a hole in the prefix, and lengths of the prefix that are none
    table0 = c.table0.copy()
    c.table0[9], c.ref = -1, None
    c.check(c.call(sv, h))
    c.table0 = table0
    for prefix in (-16, 161, 176, 2 ** 31 - 16):
        c.prefix, c.ref = prefix, None
        got = c.call(sv, h)
        c.check(got)
        assert not got["out"].any() and (got["row_status"] != 0).tolist() == [True, False, True, True, True, True]
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,hq", [(1, 8), (17, 8), (32, 16)])
def test_prefix_attention_of_not_finite_values_and_scales(sv, h, rows, hq):  # noqa: F811
    """What every row sees, it sees: an infinite key or value of the prefix; scales of either sign, and zero."""
    for where in ("k", "v"):
        c = Shared(5, "bf16", 3, rows, hq, 2, 128, 16, 320, [rows, rows + 40, 0])
        (c.kc_t if where == "k" else c.vc_t)[int(c.table0[2]), 1, 3, 7] = math.inf
        got = c.call(sv, h)
        ref = S.prefix_attention(c.q, _np(c.kc_t), _np(c.vc_t), c.tables, c.lens, c.table0, c.prefix, c.parents, c.scale)[0]
        g = _np(got["out"])
        np.testing.assert_array_equal(np.isfinite(g), np.isfinite(ref))
    c = Shared(6, "bf16", 3, rows, hq, 2, 128, 16, 320, [rows, rows + 40, 0])
    for scale in (-0.05, 0.0, 1.0):
        c.check(c.call(sv, h, scale=scale), scale)


def test_prefix_attention_is_the_same_every_time_and_on_two_streams(sv, h):  # noqa: F811
    import torch

    cases = [Shared(11 + r, "bf16", 4, r, 8, 2, 128, 16, 1600, [r, r + 100, 0, 700]) for r in (17, 1)]
    ones = [c.call(sv, h) for c in cases]
    for c, one in zip(cases, ones):
        c.check(one)
    args = [(c.args(), None if c.parents is None else _dev(c.parents)) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s, (a, p) in zip(streams, args):
            outs.append(sv.specv_prefix_attention(h, *a, parents=p, lse=True, stream=s))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        for key in ("out", "lse", "row_status"):
            assert torch.equal(out[key], ones[i % 2][key])


@pytest.mark.parametrize("rows", [1, 17])
def test_prefix_attention_in_a_captured_graph(sv, h, rows):  # noqa: F811
    """A captured call follows new lengths of the prefix and the sequences, tables and values."""
    import torch

    cases = [Shared(20 + i, "bf16", 3, rows, 8, 2, 128, 16, p, lens)
             for i, (p, lens) in enumerate(((320, [rows, 90, 0]), (0, [100, rows, rows + 1]), (1600, [0, 333, rows])))]
    blocks, width = max(c.kc_t.shape[0] for c in cases), max(c.tables.shape[1] for c in cases)
    kc = torch.zeros((blocks, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    vc, q = torch.zeros_like(kc), torch.zeros_like(cases[0].q_t)
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, lens, par = torch.zeros((3, width), **i32), torch.zeros(3, **i32), torch.zeros((3, rows - 1), **i32)
    table0, len0 = torch.zeros(100, **i32), torch.zeros(1, **i32)

    def call():
        return sv.specv_prefix_attention(h, q, kc, vc, tables, lens, table0, len0, parents=par, lse=True)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for c in cases + cases[::-1]:
        n = c.kc_t.shape[0]
        kc[:n], vc[:n] = c.kc_t, c.vc_t
        q.copy_(c.q_t)
        tables.fill_(-1)
        tables[:, :c.tables.shape[1]] = _dev(c.tables)
        lens.copy_(_dev(c.lens))
        table0[:len(c.table0)] = _dev(c.table0)
        len0.fill_(c.prefix)
        if rows > 1:
            par.copy_(_dev(c.parents))
        out["out"].fill_(math.nan)
        g.replay()
        torch.cuda.synchronize()
        c.check(out)


def test_prefix_attention_takes_slices(sv, h):  # noqa: F811
    import torch

    c = Shared(9, "bf16", 3, 17, 8, 2, 128, 16, 160, [17, 100, 0])
    one = c.call(sv, h)
    wide = torch.zeros((3, 17, 12, 128), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 1:9] = c.q_t
    pools = torch.full((c.kc_t.shape[0], 2, *c.kc_t.shape[1:]), math.nan, dtype=torch.bfloat16, device="cuda")
    pools[:, 0], pools[:, 1] = c.kc_t, c.vc_t
    a = list(c.args())
    a[0], a[1], a[2] = wide[:, :, 1:9], pools[:, 0], pools[:, 1]
    two = sv.specv_prefix_attention(h, *a, parents=_dev(c.parents), lse=True)
    assert torch.equal(one["out"], two["out"]) and torch.equal(one["lse"], two["lse"])


def test_withheld_copy_of_a_prefix_is_told(sv):  # noqa: F811
    """A copy that never lands ends the call's waits; every sequence is told, and the next call is clean."""
    hv = sv.specv_create(0, max_batch=16, max_k=31, vocab=1000)
    c = Shared(12, "bf16", 3, 17, 8, 2, 128, 16, 1600, [17, 100, 0])
    for use in (0, 1):  # the keys, the values of the one tile that a CTA has
        sv.specv_test_withhold_stage(hv, use, 2000)
        got = c.call(sv, hv)
        assert [s & 64 for s in got["row_status"].tolist()] == [64, 64, 0]
        c.check(c.call(sv, hv))
    sv.specv_destroy(hv)


def test_prefix_attention_is_refused_without_launching(sv, h):  # noqa: F811
    import torch

    c = Shared(13, "bf16", 3, 2, 8, 2, 64, 16, 32, [2, 9, 0])
    q, kc, vc, tables, lens, t0, n0 = c.args()
    before = sv.specv_launch_count(h)

    def refused(*a, **kw):
        with pytest.raises((ValueError, TypeError, sv.SpecvError)):
            sv.specv_prefix_attention(h, *a, **kw)

    refused(q, kc, vc, tables, lens, t0[None], n0)
    refused(q, kc, vc, tables, lens, t0.long(), n0)
    refused(q, kc, vc, tables, lens, t0, n0[:0])
    refused(q, kc, vc, tables, lens, t0, torch.zeros(2, dtype=torch.int32, device="cuda"))
    refused(q, kc, vc, tables, lens, t0.cpu(), n0)
    refused(q, kc, vc, tables, lens, t0, n0, scale=math.nan)
    refused(q, kc, vc, tables, lens, t0, n0, out={"out": q})
    refused(q, kc, vc, tables, lens, t0, n0, workspace=torch.zeros(1024, dtype=torch.uint8, device="cuda"))
    refused(q[:, :, :7], kc, vc, tables, lens, t0, n0)
    refused(torch.zeros((3, 33, 8, 64), dtype=torch.bfloat16, device="cuda"), kc, vc, tables, lens, t0, n0)
    assert sv.specv_launch_count(h) == before
    assert sv.specv_prefix_attention_workspace(h, sv.SPECV_BF16, 2, 64, 7, 3, 2) == 0
    assert sv.specv_prefix_attention_workspace(h, sv.SPECV_BF16, 2, 64, 8, 0, 2) == 0
    assert sv.specv_prefix_attention_workspace(h, sv.SPECV_BF16, 2, 72, 8, 3, 2) == 0
    assert sv.specv_prefix_attention_workspace(h, sv.SPECV_BF16, 2, 64, 8, 3, 2) > 0
    empty = sv.specv_prefix_attention(h, q[:0], kc, vc, tables[:0], lens[:0], t0, n0, lse=True)
    assert empty["out"].shape[0] == 0 and sv.specv_launch_count(h) == before
    # an empty pool, nothing in it: idle sequences alone
    none = kc[:0]
    got = sv.specv_prefix_attention(h, q, none, none.clone(), tables[:, :0].contiguous(), torch.zeros_like(lens), t0[:0], n0 * 0)
    assert not got["out"].any() and not got["row_status"].any()


def _exact_rows(c):
    """Outputs, sums and the bounds' ingredients in 64 bits on the GPU, a sequence at a time."""
    import torch

    B, rows, hq, dim = c.q.shape
    hkv, bs = c.kc_t.shape[1], c.bs
    outs = [torch.zeros((B, rows, hq, dim), dtype=torch.float64, device="cuda") for _ in range(2)]
    sums = [torch.zeros((B, rows, hq), dtype=torch.float64, device="cuda") for _ in range(2)]
    for b, n in enumerate(c.lens.tolist()):
        t = torch.arange(n, device="cuda")
        full = c.tables[b].copy()
        full[:c.prefix // bs] = c.table0
        blk = _dev(full).long()[t // bs]
        K, V = (x[blk, :, t % bs].double() for x in (c.kc_t, c.vc_t))
        _, _, seen = P.tree(None if c.parents is None else c.parents[b], rows)
        shut = torch.zeros((rows, n), dtype=torch.bool)
        for r in range(rows):
            shut[r, [n - rows + j for j in range(rows) if j not in seen[r]]] = True
        q = c.q_t[b].double().reshape(rows, hkv, -1, dim)
        s = (torch.einsum("rhgd,nhd->hgrn", q, K) * c.scale).masked_fill(shut.cuda(), -math.inf)
        p = torch.softmax(s, -1)
        for o, v in zip(outs, (V, V.abs())):
            o[b] = torch.einsum("hgrn,nhd->rhgd", p, v).reshape(rows, hq, dim)
        sums[0][b] = torch.logsumexp(s, -1).permute(2, 0, 1).reshape(rows, hq)
        mag = torch.einsum("rhgd,nhd->hgrn", q.abs(), K.abs()).amax(-1) * c.scale
        sums[1][b] = mag.permute(2, 0, 1).reshape(rows, hq)
    return [x.cpu().numpy() for x in (outs[0], sums[0], outs[1], sums[1])]


@pytest.mark.parametrize("B,hq,hkv,dim,bs,prefix,lens", [
    (16, 8, 2, 64, 16, 20480, [17 + 29 * i for i in range(16)]),    # row tiles of 256, the sequences beside them
    (5, 8, 2, 128, 16, 25600, [17, 600, 30, 256, 900]),             # three row tiles side by side
    (6, 24, 4, 112, 40, 20000, [40, 17, 500, 90, 1000, 120]),       # five, blocks that do not fill tiles
    (3, 16, 2, 128, 128, 384, [2000, 1500, 3000]),                  # more of their own than shared
])
def test_prefix_attention_with_both_parts_at_a_time(sv, h, B, hq, hkv, dim, bs, prefix, lens):  # noqa: F811
    c = Shared(B + prefix, "bf16", B, 17, hq, hkv, dim, bs, prefix, lens)
    got = c.call(sv, h)
    out, lse, avg, mag = _exact_rows(c)
    assert not got["row_status"].any()
    t_out, t_lse = P.attention_bounds(out, lse, avg, mag, int(c.lens.max()), dim, True)
    assert (np.abs(_np(got["out"]) - out) <= t_out).all()
    assert (np.abs(_np(got["lse"]) - lse) <= t_lse).all()
    again = c.call(sv, h)
    assert (got["out"] == again["out"]).all() and (got["lse"] == again["lse"]).all()


def test_prefix_attention_past_32_bit_offsets(sv, h):  # noqa: F811
    """A pool of more than 2^32 bytes and elements: blocks far in it, for the prefix and the sequences."""
    import torch

    bs, hkv, dim, rows = 16, 8, 128, 17
    blocks = 2 ** 32 // (bs * hkv * dim) // 2 + 600
    kc = torch.zeros((blocks, hkv, bs, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    c = Shared(77, "bf16", 3, rows, 32, hkv, dim, bs, 640, [rows, 100, 300])
    n = c.kc_t.shape[0]
    kc[-n:], vc[-n:] = c.kc_t, c.vc_t
    shift = blocks - n
    tables, table0 = _dev(c.tables + np.where(c.tables >= 0, shift, 0).astype(np.int32)), _dev(c.table0 + shift)
    for r in (rows, 1):
        q = c.q_t[:, :r].contiguous()
        lens = _dev(c.lens)
        par = _dev(c.parents) if r > 1 else None
        a = sv.specv_prefix_attention(h, q, kc, vc, tables, lens, table0, c.args()[6], parents=par, lse=True)
        b = sv.specv_prefix_attention(h, q, c.kc_t, c.vc_t, _dev(c.tables), lens, _dev(c.table0), c.args()[6], parents=par,
                                      lse=True)
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,rows,hq,hkv,dim,bs,prefix,lens", [
    (500, 1, 1, 1, 16, 3, 9, [1 + i % 7 for i in range(500)]),      # many sequences
    (8, 32, 256, 1, 64, 64, 128, [32 + 9 * i for i in range(8)]),   # 65,536 rows of one kv head
    (2, 3, 64, 64, 32, 8, 64, [3, 40]),                             # many kv heads
    (3, 17, 8, 2, 128, 1024, 1024, [17, 1024, 2000]),               # blocks longer than tiles
    (2, 32, 1, 1, 256, 16, 4096, [32, 33]),
])
def test_prefix_attention_at_the_ends_of_the_sizes(sv, h, dtype, B, rows, hq, hkv, dim, bs, prefix, lens):  # noqa: F811
    c = Shared(B + rows, dtype, B, rows, hq, hkv, dim, bs, prefix, lens)
    got = c.call(sv, h)
    out, lse, avg, mag = _exact_rows(c)
    assert not got["row_status"].any()
    t_out, t_lse = P.attention_bounds(out, lse, avg, mag, int(c.lens.max()), dim, dtype == "bf16")
    assert (np.abs(_np(got["out"]) - out) <= t_out).all()
    assert (np.abs(_np(got["lse"]) - lse) <= t_lse).all()
