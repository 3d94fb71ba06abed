"""GPU parity of append with head norms and positions on axes, gathered
attention weight and eviction with their plain float64 restatements
(serving_plain.py)."""
import math

import numpy as np
import pytest

import cache_plain as P
import serving_plain as S
from test_gpu_cache import BF16_HALF, F32_HALF, Case, _append_case, _dev, _dtype, _np, _rounded, _tables, h, sv  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------- append
# B, rows, q heads, kv heads, dim, block, lengths, tree, rot, interleaved, counts, axes, offsets
NORMS = [
    (1, 1, 1, 1, 16, 1, [1], "chain", 16, False, None, 0, False),
    (8, 1, 32, 8, 128, 16, [5, 1, 0, 900, 64, 17, 33, 2], "chain", 128, False, None, 0, True),
    (3, 17, 8, 2, 128, 16, [17, 30, 200], "tree", 128, False, None, 0, True),
    (3, 9, 6, 3, 96, 5, [9, 0, 77], "tree", 96, True, None, 0, False),
    (2, 20, 4, 2, 80, 7, [33, 20], "chain", 40, False, [20, 11], 3, False),
    (2, 7, 5, 1, 48, 16, [7, 50], "star", 6, False, None, 0, True),
    (2, 11, 3, 3, 256, 16, [40, 11], "chain", 256, False, [3, 11], 2, False),
    (2, 6, 4, 2, 256, 8, [6, 60], "chain", 128, True, None, 4, False),
    (2, 5, 2, 2, 112, 16, [5, 9], "chain", 0, False, None, 1, False),
    (2, 5, 2, 2, 144, 16, [5, 9], "chain", 22, True, [0, 5], 16, False),
    (1, 300, 4, 4, 64, 16, [310], "chain", 64, False, None, 3, False),
    (400, 3, 2, 1, 32, 3, [3 + i % 9 for i in range(400)], "chain", 32, False, None, 1, False),
]


def _norm_call(sv, h, dtype, shape, which, eps=1e-6, add=0.0):
    import torch

    B, rows, hq, hkv, dim, bs, lens, kind, rot, inter, counts, axes, shifted = shape
    rng, lens, tables, pools, xs, inv, par = _append_case(rows + dim, dtype, B, rows, hq, hkv, dim, bs, lens, kind, rot)
    weights = [_rounded(rng, (dim,), dtype) for _ in range(2)]
    counts = None if counts is None else np.array(counts, np.int32)
    pos = rng.integers(-5000, 100000, (B, rows, axes)).astype(np.int32) if axes else None
    axis = rng.integers(0, axes, rot // 2).tolist() if axes > 1 else None
    offsets = rng.integers(-300, 100000, B).astype(np.int32) if shifted else None
    w = [weights[i] if which[i] else (None, None) for i in range(2)]
    ref_k, ref_v = pools[0][1].copy(), pools[1][1].copy()
    ref = S.append_norm(ref_k, ref_v, tables, lens, xs[1][1], xs[2][1], q=xs[0][1], q_norm=w[0][1], k_norm=w[1][1], eps=eps,
                        add=add, inv_freq=inv, interleaved=inter, positions=pos, axis=axis, offsets=offsets, parents=par,
                        counts=counts)

    def call(kc, vc, **kw):
        def dev(a):
            return None if a is None else _dev(a)

        got = sv.specv_cache_append_norm(
            h, kc, vc, _dev(tables), _dev(lens), xs[1][0], xs[2][0], q=kw.pop("q", xs[0][0]), q_norm=w[0][0],
            k_norm=w[1][0], eps=eps, weight_add=add, inv_freq=dev(inv), interleaved=inter, positions=dev(pos),
            pair_axis=axis, offsets=dev(offsets), parents=dev(par), row_counts=dev(counts), **kw)
        torch.cuda.synchronize()
        return got

    return call, pools, ref, ref_k, ref_v


@pytest.mark.parametrize("which", [(True, True), (True, False), (False, True), (False, False)], ids=["qk", "q", "k", "none"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", NORMS, ids=lambda s: "B%d_R%d_H%d-%d_D%d_bs%d_rot%d_x%d" % (s[:6] + (s[8], s[11])))
def test_append_norm_matches_the_formula(sv, h, dtype, shape, which):  # noqa: F811
    add = 1.0 if shape[1] % 2 else 0.0
    call, pools, ref, ref_k, ref_v = _norm_call(sv, h, _dtype(dtype), shape, which, add=add)
    (kc_t, kc), (vc_t, _) = pools
    got = call(kc_t, vc_t)
    q_out, status, written, (q_mag, k_mag) = ref
    half = BF16_HALF if dtype == "bf16" else F32_HALF
    np.testing.assert_array_equal(got["row_status"].cpu().numpy(), status)
    np.testing.assert_array_equal(_np(vc_t), ref_v)  # values are moved, bit by bit
    kg, dim = _np(kc_t), kc.shape[-1]
    hit = np.zeros(kc.shape, bool)
    for blk, slot in written:
        hit[blk, :, slot] = True
    np.testing.assert_array_equal(kg[~hit], kc[~hit])  # nothing else is touched
    assert (np.abs(kg - ref_k) <= S.append_norm_bound(ref_k, k_mag, dim, half))[hit].all()
    gq = _np(got["q_out"])
    assert (np.abs(gq - q_out) <= S.append_norm_bound(q_out, q_mag, dim, half)).all(), np.max(np.abs(gq - q_out))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot,inter", [(128, False), (64, True), (0, False), (22, False), (22, True)])
def test_append_norm_without_more_is_append(sv, h, dtype, rot, inter):  # noqa: F811
    import torch

    rng, lens, tables, pools, xs, inv, par = _append_case(5, _dtype(dtype), 3, 9, 8, 2, 128, 16, [9, 40, 100], "tree", rot)
    (kc, _), (vc, _) = pools
    k2, v2 = kc.clone(), vc.clone()
    args = (_dev(tables), _dev(lens), xs[1][0], xs[2][0])
    kw = dict(q=xs[0][0], inv_freq=None if inv is None else _dev(inv), interleaved=inter, parents=_dev(par))
    one = sv.specv_cache_append(h, kc, vc, *args, **kw)
    two = sv.specv_cache_append_norm(h, k2, v2, *args, **kw)
    assert torch.equal(one["q_out"], two["q_out"]) and torch.equal(kc, k2) and torch.equal(vc, v2)


def test_append_norm_in_place_and_in_slices(sv, h):  # noqa: F811
    import torch

    shape = (3, 9, 6, 3, 96, 5, [9, 0, 77], "tree", 96, False, None, 0, True)
    call, pools, ref, _, _ = _norm_call(sv, h, torch.bfloat16, shape, (True, True))
    one = call(pools[0][0], pools[1][0])
    # (in place the idle sequence's rows are written over with zeros, as in other memory)
    q = _append_case(9 + 96, torch.bfloat16, 3, 9, 6, 3, 96, 5, [9, 0, 77], "tree", 96)[4][0][0]  # the call's queries
    qq = q.clone()
    two = call(pools[0][0], pools[1][0], q=qq, out={"q_out": qq})
    assert torch.equal(two["q_out"], one["q_out"]) and two["q_out"] is qq
    wide = torch.zeros((3, 9, 12, 96), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 2:8] = q
    three = call(pools[0][0], pools[1][0], q=wide[:, :, 2:8])
    assert torch.equal(three["q_out"], one["q_out"])


def test_append_norm_refuses_sequences(sv, h):  # noqa: F811
    """Nothing of a refused sequence is written, its queries are zeros; the others are done."""
    import torch

    rng, lens, tables, pools, xs, inv, par = _append_case(4, torch.float32, 7, 4, 2, 2, 32, 16,
                                                          [20, 20, 64, 20, 20, 0, 40], "tree", 32)
    lens = np.array([20, 3, 65, 20, 20, -4, 40], np.int32)
    par[3, 2], par[4, 0] = 2, -9
    tables[6, 2] = -1
    (kc_t, kc), (vc_t, vc) = pools
    w_t, w = _rounded(rng, (32,), torch.float32)
    got = sv.specv_cache_append_norm(h, kc_t, vc_t, _dev(tables), _dev(lens), xs[1][0], xs[2][0], q=xs[0][0], q_norm=w_t,
                                     k_norm=w_t, inv_freq=_dev(inv), parents=_dev(par))
    torch.cuda.synchronize()
    assert got["row_status"].tolist() == [0, 2048, 2048, 512, 512, 2048, 4096]
    q_out, status, _, (q_mag, k_mag) = S.append_norm(kc, vc, tables, lens, xs[1][1], xs[2][1], q=xs[0][1], q_norm=w,
                                                     k_norm=w, inv_freq=inv, parents=par)
    np.testing.assert_array_equal(_np(vc_t), vc)
    assert (np.abs(_np(kc_t) - kc) <= S.append_norm_bound(kc, k_mag, 32, F32_HALF)).all()
    assert (np.abs(_np(got["q_out"]) - q_out) <= S.append_norm_bound(q_out, q_mag, 32, F32_HALF)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_norm_of_zeros_and_extremes(sv, h, dtype):  # noqa: F811
    """A head of zeros stays zero (eps), tiny and large heads come out at the weight's size, one NaN or infinity takes its
    own head only."""
    import torch

    dt = _dtype(dtype)
    x = torch.ones((1, 1, 6, 64), device="cuda")
    for i, f in enumerate((0.0, 1e-12, 1e15, 1.0, 1.0, 3.0)):
        x[:, :, i] *= f
    x[0, 0, 3, 5], x[0, 0, 4, 60] = math.nan, math.inf
    kc, w = torch.zeros((1, 6, 1, 64), dtype=dt, device="cuda"), torch.full((64,), 2.0, dtype=dt, device="cuda")
    vc, one = kc.clone(), torch.ones(1, dtype=torch.int32, device="cuda")
    sv.specv_cache_append_norm(h, kc, vc, one[:, None] - 1, one, x.to(dt), x.to(dt), k_norm=w, eps=1e-6)
    k = _np(kc)[0, :, 0]
    assert (k[0] == 0).all() and np.abs(k[1] - 2e-9).max() < 2e-9 * 2.0 ** -7
    assert np.abs(k[2] - 2).max() <= 2 * 2.0 ** -8 and np.abs(k[5] - 2).max() <= 2 * 2.0 ** -8
    assert np.isnan(k[3]).all()
    assert np.isnan(k[4, 60]) and (k[4, :60] == 0).all()


# ---------------------------------------------------------------------------- mass
# B, rows, q heads, kv heads, dim, block, lengths, tree, first
MASSES = [
    (1, 1, 1, 1, 16, 1, [1], "chain", 0),
    (4, 1, 32, 8, 128, 16, [0, 1, 63, 300], "chain", 0),
    (5, 3, 6, 2, 80, 5, [3, 0, 64, 65, 131], "tree", 4),
    (3, 17, 8, 2, 128, 16, [17, 129, 400], "tree", 20),
    (2, 17, 16, 4, 96, 32, [40, 200], "star", 64),
    (2, 32, 16, 2, 128, 64, [33, 300], "line", 0),   # 256 queries a kv head: some at a time
    (2, 9, 24, 2, 256, 16, [9, 150], "tree", 3),
    (3, 31, 5, 5, 48, 3, [31, 95, 96], "tree", 1000),
    (70, 2, 4, 2, 64, 16, [2 + 5 * i for i in range(70)], "tree", 16),
    (2, 21, 4, 1, 64, 128, [21, 500], "tree", 130),  # a queries' tile more than at a time
    (2, 32, 40, 1, 128, 16, [33, 260], "tree", 0),
    (3, 7, 80, 2, 64, 8, [7, 100, 0], "star", 0),    # 280 queries
    (1, 32, 5, 1, 112, 24, [900], "tree", 5),
    (2, 25, 20, 4, 128, 40, [25, 700], "tree", 0),   # 125 queries, blocks that do not fill tiles
    (40, 1, 12, 6, 128, 16, [1 + 90 * (i % 8) for i in range(40)], "chain", 0),
    (500, 1, 2, 1, 16, 2, [1 + i % 9 for i in range(500)], "chain", 1),
    (2, 2, 64, 64, 32, 8, [40, 300], "chain", 0),    # many kv heads
    (2, 5, 8, 2, 64, 1024, [1500, 2048], "tree", 1024),
]


def _mass_case(seed, dtype, shape):
    B, rows, hq, hkv, dim, bs, lens, kind, first = shape
    c = Case(seed, dtype, B, rows, hq, hkv, dim, bs, lens, kind)
    _, lse, _, _, _ = P.attention(c.q, _np(c.kc_t), _np(c.vc_t), c.tables, c.lens, c.parents, c.scale)
    c.lse = np.where(np.isfinite(lse), lse, 0).astype(np.float32)
    return c


def _mass_check(c, got, before, first, lse, old, scale=None):
    ref, status, written, tol = S.mass(c.q, _np(c.kc_t), c.tables, c.lens, lse, c.parents,
                                       c.scale if scale is None else scale, before, first, got["mass"].shape[-1])
    np.testing.assert_array_equal(got["row_status"].cpu().numpy(), status)
    g = _np(got["mass"])
    np.testing.assert_array_equal(g[~written], np.broadcast_to(old, g.shape)[~written])  # nothing else is touched
    bad = written & ~(np.abs(g - ref) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4], g[bad][:4], ref[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", MASSES, ids=lambda s: "B%d_R%d_H%d-%d_D%d_bs%d_first%d" % (s[:6] + (s[8],)))
def test_mass_matches_the_formula(sv, h, dtype, shape):  # noqa: F811
    import torch

    c, first = _mass_case(3, dtype, shape), shape[8]
    par = None if c.parents is None else _dev(c.parents)
    width = c.tables.shape[1] * shape[5] + 3
    args = (h, c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), _dev(c.lse))
    got = sv.specv_attention_mass(*args, first=first, parents=par)
    torch.cuda.synchronize()
    _mass_check(c, got, None, first, c.lse, 0.0)
    before = c.rng.random((shape[0], shape[3], width)).astype(np.float32)
    # what the pass's own positions held, and what lies before and behind, has no say
    clean = before.copy()
    for b, n in enumerate(c.lens):
        before[b, :, max(int(n) - shape[1], 0):] = np.nan
    out = torch.full((shape[0], shape[3], width), -7.0, device="cuda")
    got = sv.specv_attention_mass(*args, mass=_dev(before), first=first, parents=par, out={"mass": out})
    torch.cuda.synchronize()
    assert got["mass"] is out
    _mass_check(c, got, before, first, c.lse, -7.0)
    both = _dev(clean)
    sv.specv_attention_mass(*args, mass=both, first=first, parents=par, out={"mass": both})  # in place
    got = sv.specv_attention_mass(*args, mass=_dev(clean), first=first, parents=par)
    torch.cuda.synchronize()
    _, _, written, _ = S.mass(c.q, c.kc, c.tables, c.lens, c.lse, c.parents, c.scale, None, first, width)
    w = _dev(written)
    assert torch.equal(both[w], got["mass"][w]) and torch.equal(both[~w], _dev(clean)[~w])


@pytest.mark.parametrize("rows,hq", [(1, 8), (5, 8), (17, 8), (32, 16)])
def test_mass_of_attention_adds_up_to_the_rows(sv, h, rows, hq):  # noqa: F811
    """With the attention's own sums, each row and head hands out a weight of one; a row of infinite lse none; a negative
    scale and a long cache alike."""
    import torch

    c = Case(7, "bf16", 3, rows, hq, 2, 128, 16, [rows, 3000, 517], "tree")
    par = None if c.parents is None else _dev(c.parents)
    for scale in (c.scale, -0.02):
        args = (h, c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens))
        att = sv.specv_tree_attention(*args, parents=par, lse=True, scale=scale)
        got = sv.specv_attention_mass(*args, att["lse"], parents=par, scale=scale)
        torch.cuda.synchronize()
        assert (got["mass"].double().sum(-1) - rows * hq / 2).abs().max() < rows * hq * 2.0 ** -14
        _mass_check(c, got, None, 0, _np(att["lse"]), 0.0, scale)
        lse = att["lse"].clone()
        lse[:, 0], lse[1] = math.inf, math.inf
        got = sv.specv_attention_mass(*args, lse, parents=par, scale=scale)
        torch.cuda.synchronize()
        _mass_check(c, got, None, 0, _np(lse), 0.0, scale)
        assert not got["mass"][1].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hq", [(2, 2), (17, 4)])
def test_mass_of_hidden_and_infinite_keys(sv, h, dtype, rows, hq):  # noqa: F811
    """A hidden key that is NaN or infinite gathers from its own row's path alone and changes no other position."""
    import torch

    c = Case(8, dtype, 1, rows, hq, 1, 64, 16, [150], "star")
    want = _mass_case(8, dtype, (1, rows, hq, 1, 64, 16, [150], "star", 0)).lse
    args = (h, c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), _dev(want))
    par = None if c.parents is None else _dev(c.parents)
    clean = sv.specv_attention_mass(*args, parents=par)["mass"].clone()
    t = 149  # the last row's own key: no other row sees it
    blk, slot = int(c.tables[0, t // 16]), t % 16
    for x in (math.nan, math.inf):
        c.kc_t[blk, 0, slot, 3] = x
        got = sv.specv_attention_mass(*args, parents=par)["mass"]
        assert torch.equal(got[..., :t], clean[..., :t])
        assert x == math.inf or torch.isnan(got[0, 0, t])


@pytest.mark.parametrize("dtype,rows,hq,first",
                         [("bf16", 17, 8, 0), ("bf16", 6, 8, 197), ("f32", 9, 4, 194), ("bf16", 32, 24, 0), ("f32", 32, 8, 0)])
def test_mass_of_a_verified_pass(sv, h, dtype, rows, hq, first):  # noqa: F811
    """Rejected rows give nothing, kept nodes' masses go along the path; a path or count that is none is refused."""
    import torch

    B, lens = 6, [rows, 150, 0, 200, 130, 131]  # (`first` of 197 and 194: inside the pass of the fourth)
    c = _mass_case(rows, dtype, (B, rows, hq, 2, 64, 16, lens, "star", first))
    M = rows - 1
    acc = np.array([0, M, 1, M // 2, M + 1, 2], np.int32)
    path = np.full((B, M), -1, np.int32)
    for b in range(B):
        path[b, :min(acc[b], M)] = np.sort(c.rng.permutation(M)[:min(acc[b], M)])
    path[5, :2] = path[5, 1::-1]  # not increasing
    width = c.tables.shape[1] * 16
    for p in (path, None):
        before = c.rng.random((B, 2, width)).astype(np.float32)
        out = torch.full((B, 2, width), -7.0, device="cuda")
        got = sv.specv_attention_mass(h, c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), _dev(c.lse), mass=_dev(before),
                                      first=first, parents=_dev(c.parents), path=None if p is None else _dev(p),
                                      num_accepted=_dev(acc), out={"mass": out})
        torch.cuda.synchronize()
        ref, status, written, tol = S.mass(c.q, _np(c.kc_t), c.tables, c.lens, c.lse, c.parents, c.scale, before, first, width,
                                           p, acc)
        assert got["row_status"].tolist() == status.tolist()
        # (of a sequence within the whole blocks before `first` only the length is looked at)
        assert status.tolist()[4:] == ([0, 0] if first >= lens[5] else [128, 0 if p is None else 8192])
        g = _np(out)
        assert (g[~written] == -7.0).all() and (np.abs(g - ref) <= tol)[written].all()


def test_mass_refuses_sequences(sv, h):  # noqa: F811
    import torch

    c = _mass_case(5, "bf16", (8, 4, 8, 2, 64, 16, [20, 20, 64, 20, 40, 30, 0, 50], "tree", 0))
    c.lens[:] = [20, 3, 65, 20, 40, -1, 0, 50]
    c.parents[3, 2] = 2
    c.tables[4, 0] = 10 ** 6
    out = torch.full((8, 2, 64), -7.0, device="cuda")
    got = sv.specv_attention_mass(h, c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), _dev(c.lse),
                                  parents=_dev(c.parents), out={"mass": out})
    torch.cuda.synchronize()
    assert got["row_status"].tolist() == [0, 2048, 2048, 512, 4096, 2048, 0, 0]
    _mass_check(c, got, None, 0, c.lse, -7.0)
    narrow = sv.specv_attention_mass(h, c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), _dev(c.lse),
                                     parents=_dev(c.parents), out={"mass": torch.zeros((8, 2, 49), device="cuda")})
    assert narrow["row_status"].tolist() == [0, 2048, 2048, 512, 4096, 2048, 0, 2048]


# ---------------------------------------------------------------------------- eviction
# B, layers, heads, dim, block, lengths, budget, recent, first
EVICTS = [
    (1, 1, 1, 16, 1, [3], 1, 0, 0),
    (4, 1, 2, 64, 16, [0, 40, 41, 200], 40, 8, 0),
    (3, 2, 8, 128, 16, [300, 100, 129], 100, 30, 4),
    (2, 3, 3, 80, 5, [77, 1], 30, 0, 7),
    (2, 1, 1, 256, 64, [500, 640], 128, 127, 0),      # nearly all recent
    (2, 1, 2, 48, 3, [90, 91], 40, 25, 15),           # no place for any other
    (2, 1, 4, 128, 16, [1500, 2600], 1300, 64, 16),   # more moves than are listed at a time
    (1, 2, 1, 96, 16, [6000], 3000, 10, 0),
    (80, 1, 8, 64, 16, [20 + i for i in range(80)], 50, 20, 2),
    (3, 40, 8, 32, 8, [30, 29, 64], 29, 5, 1),
    (1, 1, 2, 16, 256, [30000], 17000, 3000, 100),    # many spans of masses, many lists of moves
    (500, 1, 1, 16, 2, [3 + i % 11 for i in range(500)], 6, 2, 1),
]


@pytest.mark.parametrize("masses", ["spread", "ties", "odd"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", EVICTS, ids=lambda s: "B%d_L%d_H%d_D%d_bs%d_to%d-%d-%d" % (s[:5] + s[6:]))
def test_eviction_matches(sv, h, dtype, shape, masses):  # noqa: F811
    import torch

    B, layers, heads, dim, bs, lens, budget, recent, first = shape
    rng = np.random.default_rng(budget + dim)
    lens = np.array(lens, np.int32)
    tables, blocks = _tables(rng, lens, bs)
    pools = [_rounded(rng, (layers, blocks, heads, bs, dim), _dtype(dtype)) for _ in range(2)]
    width = tables.shape[1] * bs + 5
    m = rng.exponential(size=(layers, B, heads, width)) ** 3
    if masses == "ties":
        m = np.floor(m * 2) / 4
    if masses == "odd":  # zeros of both signs, negative masses, infinities, what is no number, the smallest there are
        odd = np.array([0.0, -0.0, -1.5, math.inf, -math.inf, math.nan, 1e-45, 2e-45, 1.0])
        m = np.where(rng.random(m.shape) < 0.7, odd[rng.integers(0, len(odd), m.shape)], m)
    m = m.astype(np.float32)
    ref = [p[1].copy() for p in pools]
    places, new, status = S.evict(*ref, tables, lens, m, budget, recent, first)
    kc, vc = pools[0][0], pools[1][0]
    if layers == 1:
        kc, vc = kc[0], vc[0]
    m_t = _dev(m if layers > 1 else m[0])
    out = torch.full_like(m_t, -7.0)
    got = sv.specv_cache_evict(h, kc, vc, _dev(tables), _dev(lens), m_t, budget, recent=recent, first=first,
                               out={"mass": out})
    torch.cuda.synchronize()
    assert got["row_status"].tolist() == status.tolist() and got["seq_lens"].tolist() == new.tolist()
    assert got["evicted"].tolist() == (lens - new).tolist()
    np.testing.assert_array_equal(_np(pools[0][0]), ref[0])
    np.testing.assert_array_equal(_np(pools[1][0]), ref[1])
    g = out.cpu().numpy().reshape(m.shape)
    want = np.full_like(m, -7.0)
    for b in range(B):
        for l in range(layers):
            for hh in range(heads):
                place = places[l][b][hh]
                place = list(range(lens[b])) if place is None else place
                want[l, b, hh, :len(place)] = m[l, b, hh, place]
    np.testing.assert_array_equal(g, want)


def test_eviction_of_strided_pools_and_interleaved_layers(sv, h):  # noqa: F811
    import torch

    rng = np.random.default_rng(1)
    lens = np.array([100, 70], np.int32)
    tables, blocks = _tables(rng, lens, 16)
    pool_t, _ = _rounded(rng, (blocks, 3, 2, 4, 16, 64), torch.bfloat16)  # layers inside blocks, keys beside values
    kc, vc = pool_t[:, :, 0].transpose(0, 1), pool_t[:, :, 1].transpose(0, 1)
    ref = [_np(kc), _np(vc)]
    m = rng.random((3, 2, 4, 112)).astype(np.float32)
    S.evict(*ref, tables, lens, m, 40, 9, 3)
    got = sv.specv_cache_evict(h, kc, vc, _dev(tables), _dev(lens), _dev(m), 40, recent=9, first=3)
    torch.cuda.synchronize()
    assert got["seq_lens"].tolist() == [40, 40] and (got["mass"][..., 40:] == 0).all()
    np.testing.assert_array_equal(_np(kc), ref[0])
    np.testing.assert_array_equal(_np(vc), ref[1])


def test_eviction_refuses_sequences(sv, h):  # noqa: F811
    import torch

    rng = np.random.default_rng(2)
    lens = np.array([40, 40, 40, 40, 40, 8], np.int32)
    tables, blocks = _tables(rng, lens, 8)
    lens[:] = [40, -2, 41, 40, 40, 8]
    tables[3, 4], tables[4, 0], tables[5, 0] = blocks, -1, -5  # the last is within its budget, the one before it in front
    pools = [_rounded(rng, (1, blocks, 2, 8, 32), torch.float32) for _ in range(2)]
    ref = [p[1].copy() for p in pools]
    m = rng.random((1, 6, 2, 40)).astype(np.float32)
    places, new, status = S.evict(*ref, tables, lens, m, 20, 4, 8)
    got = sv.specv_cache_evict(h, pools[0][0][0], pools[1][0][0], _dev(tables), _dev(lens), _dev(m[0]), 20, recent=4, first=8)
    torch.cuda.synchronize()
    assert got["row_status"].tolist() == status.tolist() == [0, 2048, 2048, 4096, 0, 0]
    assert got["seq_lens"].tolist() == new.tolist() == [20, -2, 41, 40, 20, 8]
    np.testing.assert_array_equal(_np(pools[0][0]), ref[0])
    np.testing.assert_array_equal(_np(pools[1][0]), ref[1])
    got = sv.specv_cache_evict(h, pools[0][0][0], pools[1][0][0], _dev(tables), _dev(lens), _dev(m[0, :, :, :39].copy()), 64)
    assert got["row_status"].tolist() == [2048, 2048, 2048, 2048, 2048, 0]


# ---------------------------------------------------------------------------- refusals
def test_serving_calls_are_refused_without_launching(sv, h):  # noqa: F811
    import torch

    i32 = dict(dtype=torch.int32, device="cuda")
    kc, vc = torch.zeros((4, 2, 16, 64), device="cuda"), torch.zeros((4, 2, 16, 64), device="cuda")
    tables, lens = torch.zeros((2, 2), **i32), torch.zeros(2, **i32)
    k, q = torch.zeros((2, 3, 2, 64), device="cuda"), torch.zeros((2, 3, 4, 64), device="cuda")
    inv, w = torch.ones(32, device="cuda"), torch.ones(64, device="cuda")
    pos, off, par = torch.zeros((2, 3, 3), **i32), torch.zeros(2, **i32), torch.full((2, 2), -1, **i32)
    lse, mass = torch.zeros((2, 3, 4), device="cuda"), torch.zeros((2, 2, 32), device="cuda")
    before = sv.specv_launch_count(h)

    def refused(call, *a, **kw):
        with pytest.raises((ValueError, TypeError, sv.SpecvError)):
            call(h, *a, **kw)

    def append(**kw):
        refused(sv.specv_cache_append_norm, kc, vc, tables, lens, k, k, **kw)

    for kw in (dict(q_norm=w, eps=-1.0), dict(k_norm=w, eps=math.nan), dict(k_norm=w, weight_add=math.inf),
               dict(k_norm=w[:32]), dict(k_norm=w.double()), dict(k_norm=w.cpu()),
               dict(q_norm=torch.ones(65, device="cuda")[1:]), dict(k_norm=torch.ones(66, device="cuda")[2:]),
               dict(positions=pos, inv_freq=inv), dict(positions=pos, inv_freq=inv, pair_axis=[0] * 31),
               dict(positions=pos, inv_freq=inv, pair_axis=[0] * 31 + [3]), dict(pair_axis=[0] * 32, inv_freq=inv),
               dict(positions=pos, pair_axis=[0] * 32, inv_freq=inv, offsets=off),
               dict(positions=pos, pair_axis=[0] * 32, inv_freq=inv, parents=par),
               dict(positions=pos[:, :2], inv_freq=inv, pair_axis=[0] * 32), dict(offsets=off[:1]),
               dict(positions=pos.long(), inv_freq=inv, pair_axis=[0] * 32),
               dict(positions=torch.zeros((2, 3, 17), **i32), inv_freq=inv, pair_axis=[0] * 32),
               dict(positions=torch.zeros((2, 3, 0), **i32), inv_freq=inv, pair_axis=[0] * 32)):
        append(**kw)
    m = sv.specv_attention_mass
    refused(m, q[:, :, :3], kc, vc, tables, lens, lse[:, :, :3].contiguous())
    refused(m, q, kc, vc, tables, lens, lse, first=-1)
    refused(m, q, kc, vc, tables, lens, lse, path=par)
    refused(m, q, kc, vc, tables, lens, lse, path=par[:, :1], num_accepted=off)
    refused(m, q, kc, vc, tables, lens, lse, num_accepted=off[:1])
    refused(m, q, kc, vc, tables, lens, lse, scale=math.inf)
    refused(m, q, kc, vc, tables, lens, lse[:1])
    refused(m, q, kc, vc, tables, lens, lse, mass=mass[:, :1])
    long = torch.zeros((3, 2, 32), device="cuda")
    refused(m, q, kc, vc, tables, lens, lse, mass=long[:2], out={"mass": long[1:]})
    refused(m, q, kc, vc, tables, lens, lse, mass=mass, out={"mass": torch.zeros((2, 2, 31), device="cuda")})
    refused(m, torch.zeros((2, 33, 4, 64), device="cuda"), kc, vc, tables, lens, torch.zeros((2, 33, 4), device="cuda"))
    e = sv.specv_cache_evict
    for kw in (dict(budget=0), dict(budget=-3), dict(budget=4, recent=5), dict(budget=4, recent=3, first=2),
               dict(budget=4, recent=-1), dict(budget=4, first=-1), dict(budget=4, out={"mass": mass}),
               dict(budget=4, out={"seq_lens": lens})):
        refused(e, kc, vc, tables, lens, mass, kw.pop("budget"), **kw)
    both = torch.zeros((3, 2, 32), device="cuda")
    refused(e, kc, vc, tables, lens, both[:2], 4, out={"mass": both[1:]})
    refused(e, kc, vc, tables, lens, mass[0], 4)
    refused(e, kc, vc, tables, lens, mass.double(), 4)
    assert sv.specv_launch_count(h) == before


def test_serving_calls_of_empty_batches_and_pools(sv, h):  # noqa: F811
    import torch

    i32 = dict(dtype=torch.int32, device="cuda")
    kc = torch.zeros((0, 2, 16, 64), device="cuda")
    for B in (0, 3):
        tables, lens = torch.zeros((B, 0), **i32), torch.zeros(B, **i32)
        k, q = torch.zeros((B, 3, 2, 64), device="cuda"), torch.ones((B, 3, 4, 64), device="cuda")
        got = sv.specv_cache_append_norm(h, kc, kc.clone(), tables, lens, k, k, q=q, q_norm=torch.ones(64, device="cuda"))
        assert not got["q_out"].any() and not got["row_status"].any()
        got = sv.specv_attention_mass(h, q, kc, kc.clone(), tables, lens, torch.zeros((B, 3, 4), device="cuda"))
        assert got["mass"].shape == (B, 2, 0) and not got["row_status"].any()
        got = sv.specv_cache_evict(h, kc, kc.clone(), tables, lens, got["mass"], 5)
        assert not got["row_status"].any() and not got["seq_lens"].any()


# ---------------------------------------------------------------------------- together
def test_serving_calls_in_one_captured_graph(sv):  # noqa: F811
    """Append with norms, attention over a shared prefix, the weight gathered and the eviction in one graph, replayed with
    other lengths, tables and values; each replay gives what the calls one by one give."""
    import torch

    B, rows, hq, hkv, dim, bs, width, prefix = 3, 9, 8, 2, 64, 16, 20, 32
    hv = sv.specv_create(0, max_batch=B, max_k=31, vocab=100)
    i32 = dict(dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(8)
    inv = _dev((10000.0 ** (-np.arange(dim // 2) * 2 / dim)).astype(np.float32))
    w = _rounded(rng, (dim,), torch.bfloat16)[0]
    kc, vc = (torch.zeros((70, hkv, bs, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fused = torch.zeros((B, rows, hq + 2 * hkv, dim), dtype=torch.bfloat16, device="cuda")
    tables, lens, off, par = torch.zeros((B, width), **i32), torch.zeros(B, **i32), torch.zeros(B, **i32), torch.zeros((B, rows - 1), **i32)
    table0, len0 = torch.zeros(2, **i32), torch.full((1,), prefix, **i32)
    mass = torch.zeros((B, hkv, width * bs), device="cuda")

    def calls():
        q, k, v = fused[:, :, :hq], fused[:, :, hq:hq + hkv], fused[:, :, hq + hkv:]
        app = sv.specv_cache_append_norm(hv, kc, vc, tables, lens, k, v, q=q, q_norm=w, k_norm=w, inv_freq=inv, offsets=off,
                                         parents=par)
        att = sv.specv_prefix_attention(hv, app["q_out"], kc, vc, tables, lens, table0, len0, parents=par, lse=True)
        got = sv.specv_attention_mass(hv, app["q_out"], kc, vc, tables, lens, att["lse"], mass=mass, first=prefix, parents=par)
        ev = sv.specv_cache_evict(hv, kc, vc, tables, lens, got["mass"], 96, recent=20, first=prefix)
        return app["q_out"], att["out"], att["lse"], got["mass"], ev["mass"], ev["seq_lens"], ev["evicted"], ev["row_status"]

    def fill(seed):
        r = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (kc, vc, fused):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        mass.copy_(torch.rand(mass.shape, generator=g, device="cuda"))
        order = r.permutation(70)
        full = np.array([np.concatenate((order[:2], order[2 + 20 * b:20 + 20 * b])) for b in range(B)], np.int32)
        tables.copy_(_dev(full))
        table0.copy_(_dev(order[:2].astype(np.int32)))
        lens.copy_(_dev(np.array([prefix + rows, 288 if seed % 2 else 0, int(r.integers(100, 280))], np.int32)))
        off.copy_(_dev(r.integers(0, 999, B).astype(np.int32)))
        par.copy_(_dev(np.array([[r.integers(-1, i) for i in range(rows - 1)] for _ in range(B)], np.int32)))

    fill(0)
    calls()
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(calls())
    for seed in (1, 2, 3):
        fill(seed)
        want = [x.clone() for x in (*calls(), kc, vc)]
        for g, out in zip(graphs, outs):
            fill(seed)
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip((*out, kc, vc), want):
                assert torch.equal(x, y)
    sv.specv_destroy(hv)


def test_serving_calls_on_two_streams(sv, h):  # noqa: F811
    """Calls in flight together on two streams keep apart."""
    import torch

    cs = [_mass_case(40 + i, d, (4, r, 8, 2, 64, 16, [500, 40, 0, 900], "tree", 0)) for i, (d, r) in enumerate((("bf16", 9), ("f32", 3)))]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    pools = [[(c.kc_t.clone(), c.vc_t.clone()) for _ in range(4)] for c in cs]
    args = [(_dev(c.tables), _dev(c.lens), _dev(c.lse), _dev(c.parents), _dev(c.rng.random((4, 2, 960)).astype(np.float32)))
            for c in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for k in range(4):
        for i, (c, s) in enumerate(zip(cs, streams)):
            t, n, l, p, m = args[i]
            a = sv.specv_attention_mass(h, c.q_t, *pools[i][k], t, n, l, mass=m, parents=p, stream=s)
            e = sv.specv_cache_evict(h, *pools[i][k], t, n, a["mass"], 100, recent=30, first=4, stream=s)
            got[i].append((a["mass"], e["mass"], e["seq_lens"], *pools[i][k]))
    torch.cuda.synchronize()
    for i, c in enumerate(cs):
        t, n, l, p, m = args[i]
        kc, vc = c.kc_t.clone(), c.vc_t.clone()
        a = sv.specv_attention_mass(h, c.q_t, kc, vc, t, n, l, mass=m, parents=p)
        e = sv.specv_cache_evict(h, kc, vc, t, n, a["mass"], 100, recent=30, first=4)
        for one in got[i]:
            for x, y in zip(one, (a["mass"], e["mass"], e["seq_lens"], kc, vc)):
                assert torch.equal(torch.nan_to_num(x.double()), torch.nan_to_num(y.double()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_mass_of_a_long_cache_past_32_bit_offsets(sv, h, dtype):  # noqa: F811
    """Blocks far in a pool of more than 2^32 bytes, a long context, with the last position's mass at the end of a wide row."""
    import torch

    rng = np.random.default_rng(4)
    bs, hkv, dim, n, rows = 16, 4, 128, 40000, 3
    dt = _dtype(dtype)
    blocks = 2 ** 32 // (bs * hkv * dim * dt.itemsize) + 2600
    kc = torch.zeros((blocks, hkv, bs, dim), dtype=dt, device="cuda")
    used = -(-n // bs)
    tables = np.full((1, used), -1, np.int32)
    tables[0] = blocks - 1 - rng.permutation(used)
    g = torch.Generator(device="cuda").manual_seed(1)
    kc[blocks - used:] = torch.randn((used, hkv, bs, dim), generator=g, device="cuda").to(dt)
    q = (torch.randn((1, rows, 8, dim), generator=g, device="cuda") * 2).to(dt)
    lens = _dev(np.array([n], np.int32))
    att = sv.specv_tree_attention(h, q, kc, kc, _dev(tables), lens, lse=True)
    got = sv.specv_attention_mass(h, q, kc, kc, _dev(tables), lens, att["lse"])["mass"]
    t = torch.arange(n, device="cuda")
    K = kc[_dev(tables).long()[0][t // bs], :, t % bs].double()
    s = torch.einsum("rhgd,nhd->hgrn", q[0].double().reshape(rows, hkv, 2, dim), K) * dim ** -0.5
    late = t[None] > n - rows + torch.arange(rows, device="cuda")[:, None]
    s.masked_fill_(late, -math.inf)
    want = torch.exp(s - att["lse"][0].double().reshape(rows, hkv, 2).permute(1, 2, 0)[..., None]).sum((1, 2))
    # each weight is off by 2^-23 of (dim + 16) times the magnitudes (below 60), its arguments' and the exponential's rounding
    assert ((got[0, :, :n].double() - want).abs() <= want * (144 * 60 + 200) * 2.0 ** -23 + 1e-30).all()


def test_a_bounded_cache_of_all_of_them(sv):  # noqa: F811
    """Rounds of append with norms, attention over a shared prefix, verification's kept chain, the gathered weight, and
    eviction with the blocks given back, against a dense history in 64 bits: each head holds what it should hold."""
    import torch

    B, M, hq, hkv, dim, bs, prefix, budget, recent = 3, 5, 4, 2, 64, 4, 16, 40, 12
    rng = np.random.default_rng(21)
    hv = sv.specv_create(0, max_batch=B, max_k=M, vocab=60)
    inv = (10000.0 ** (-np.arange(dim // 2) * 2 / dim)).astype(np.float32)
    w_t, w = _rounded(rng, (dim,), torch.float32)
    blocks = 200
    kc = torch.zeros((blocks, hkv, bs, dim), device="cuda")
    vc = torch.zeros_like(kc)
    free = [int(x) for x in rng.permutation(blocks)]
    n0 = prefix // bs
    table0 = [free.pop() for _ in range(n0)]
    tables = np.full((B, 40), -1, np.int32)
    tables[:, :n0] = table0
    nb, lens, off = [n0] * B, np.full(B, prefix, np.int32), np.zeros(B, np.int32)
    free_list, free_count = torch.zeros(blocks, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    # the prefix, appended once
    (k_t, k), (v_t, v) = [_rounded(rng, (1, prefix, hkv, dim), torch.float32) for _ in range(2)]
    sv.specv_cache_append_norm(hv, kc, vc, _dev(tables[:1]), _dev(lens[:1]), k_t, v_t, k_norm=w_t, inv_freq=_dev(inv))
    turned = lambda x, p, wt: S.turn(S.norm(x, wt, 1e-6, 0.0), p * inv.astype(np.float64), False)  # noqa: E731
    # by sequence and head: keys, values, positions as tokens, masses, in cache order
    hist = [[[(turned(k[0, t], t, w)[h_], v[0, t, h_], t, 0.0) for t in range(prefix)] for h_ in range(hkv)] for _ in range(B)]
    mass = torch.zeros((B, hkv, 160), device="cuda")
    spare = torch.zeros_like(mass)
    for step in range(12):
        for b in range(B):
            lens[b] += M + 1
            while nb[b] * bs < lens[b]:
                tables[b, nb[b]] = free.pop()
                nb[b] += 1
        (q_t, q), (k_t, k), (v_t, v) = [_rounded(rng, (B, M + 1, n, dim), torch.float32) for n in (hq, hkv, hkv)]
        t_t, l_t = _dev(tables), _dev(lens)
        app = sv.specv_cache_append_norm(hv, kc, vc, t_t, l_t, k_t, v_t, q=q_t, q_norm=w_t, k_norm=w_t, inv_freq=_dev(inv),
                                         offsets=_dev(off))
        att = sv.specv_prefix_attention(hv, app["q_out"], kc, vc, t_t, l_t, _dev(np.array(table0, np.int32)),
                                        _dev(np.array([prefix], np.int32)), lse=True)
        accepted = rng.integers(0, M + 1, B).astype(np.int32)
        sv.specv_attention_mass(hv, app["q_out"], kc, vc, t_t, l_t, att["lse"], mass=mass, first=prefix,
                                num_accepted=_dev(accepted), out={"mass": mass})  # rejected drafts gather nothing
        for b in range(B):
            base = len(hist[b][0])
            for h_ in range(hkv):
                for r in range(M + 1):
                    hist[b][h_].append((turned(k[b, r], base + off[b] + r, w)[h_], v[b, r, h_], base + int(off[b]) + r, 0.0))
            gained = np.zeros((hkv, base + M + 1))
            for r in range(M + 1):
                qq = turned(q[b, r], base + off[b] + r, w)
                for hh in range(hq):
                    seen = hist[b][hh // 2][:base + r + 1]
                    s = np.array([x[0] for x in seen]) @ qq[hh] * dim ** -0.5
                    e = np.exp(s - s.max())
                    o = e @ np.array([x[1] for x in seen]) / e.sum()
                    # as in the verify round of the other cache calls: fp32 throughout
                    assert np.max(np.abs(_np(att["out"][b, r, hh]) - o)) < 2e-3 * max(np.abs(x[1]).max() for x in seen)
                    if r <= accepted[b]:
                        gained[hh // 2, :base + r + 1] += e / e.sum()
            for h_ in range(hkv):
                hist[b][h_] = [(x[0], x[1], x[2], x[3] + (gained[h_, t] if t >= prefix else 0.0)) for t, x in enumerate(hist[b][h_])]
                stay = len(hist[b][h_]) - (M - int(accepted[b]))
                got = _np(mass[b, h_, :stay])
                assert np.max(np.abs(got - [x[3] for x in hist[b][h_][:stay]])[prefix:]) < 1e-3
        # the rejected drafts leave, with their blocks
        nb_t, acc_t = _dev(np.array(nb, np.int32)), _dev(accepted)
        free_count.zero_()
        sv.specv_rollback(hv, acc_t, M, l_t, t_t, nb_t, bs, free_list, free_count)
        free.extend(free_list[:int(free_count)].tolist())
        ev = sv.specv_cache_evict(hv, kc, vc, t_t, l_t, mass, budget, recent=recent, first=prefix, out={"mass": spare})
        mass, spare = spare, mass
        off += ev["evicted"].cpu().numpy()
        free_count.zero_()
        new = ev["seq_lens"]
        sv.specv_rollback(hv, torch.full((B,), M, dtype=torch.int32, device="cuda"), M, new, t_t, nb_t, bs, free_list, free_count)
        free.extend(free_list[:int(free_count)].tolist())
        tables, nb, lens = t_t.cpu().numpy().copy(), nb_t.tolist(), new.cpu().numpy().copy()
        assert all(n == -(-int(x) // bs) for n, x in zip(nb, lens)) and max(lens) <= budget
        for b in range(B):
            for h_ in range(hkv):
                rows_ = hist[b][h_][:len(hist[b][h_]) - (M - int(accepted[b]))]
                if len(rows_) > budget:
                    line = budget - recent
                    got = _np(spare[b, h_, :len(rows_)])  # ties in 64 bits could fall either way: the kernel's own masses decide
                    mid = range(prefix, len(rows_) - recent)
                    kept = set(sorted(mid, key=lambda t: (-got[t], t))[:line - prefix])
                    holes = [t for t in range(prefix, line) if t not in kept]
                    above = [t for t in range(line, len(rows_) - recent) if t in kept]
                    place = list(range(line)) + list(range(len(rows_) - recent, len(rows_)))
                    for t, x in zip(holes, above):
                        place[t] = x
                    rows_ = [rows_[t] for t in place]
                hist[b][h_] = rows_
                assert len(rows_) == lens[b]
                t = np.arange(lens[b])
                ids = tables[b][t // bs]
                assert np.max(np.abs(_np(kc)[ids, h_, t % bs] - [x[0] for x in rows_])) < 2.0 ** -18
                np.testing.assert_array_equal(_np(vc)[ids, h_, t % bs], [x[1] for x in rows_])
    assert (off > 0).all()
    sv.specv_destroy(hv)
