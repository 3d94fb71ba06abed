"""The calls on the paged KV cache at the ends of the type: infinities and
the largest finite values in keys and values, seen and hidden, padding, and scales at
the ends of fp32."""
import math

import numpy as np
import pytest

import cache_plain as P
from test_gpu_cache import Case, _dev, _dtype, _np, _rounded, _tables, h, sv  # noqa: F401  (h and sv are fixtures)

pytestmark = pytest.mark.gpu

F32_MAX = float(np.finfo(np.float32).max)
# rows, query heads of two kv heads: row tiles of 16, 32 and more rows a kv head
MANY = [(3, 4), (6, 8), (17, 8), (32, 16)]


def _set(c, pool, b, t, head, col, value):
    pool[int(c.tables[b, t // 16]), head, t % 16, col] = value


@pytest.mark.parametrize("rows,hq", MANY)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_f32_values_that_a_tree_hides(sv, h, rows, hq, dim):  # noqa: F811
    """The largest and the lowest finite floats, which the nearest number of
    11 bits is infinite for, and infinities, in the last node of a star: its
    own rows alone see them."""
    c = Case(rows + dim, "f32", 2, rows, hq, 2, dim, 16, [rows, rows + 100], "star")
    for b, n in enumerate(c.lens):
        for col, val in ((0, F32_MAX), (5, -F32_MAX), (9, 3.4028e38), (11, math.inf)):
            _set(c, c.vc_t, b, int(n) - 1, 0, col, val)
        for col, val in ((0, F32_MAX), (1, -F32_MAX), (2, math.inf)):
            _set(c, c.kc_t, b, int(n) - 1, 1, col, val)
    got = c.call(sv, h)
    clean = Case(rows + dim, "f32", 2, rows, hq, 2, dim, 16, [rows, rows + 100], "star")
    out, lse, status, avg, mag = P.attention(clean.q, _np(clean.kc_t), _np(clean.vc_t), clean.tables, clean.lens,
                                             clean.parents, clean.scale)
    t_out, t_lse = P.attention_bounds(out, lse, avg, mag, int(c.lens.max()), dim, False)
    hidden = slice(0, rows - 1)  # the rows that do not see the last node
    assert got["row_status"].tolist() == [0, 0]
    assert (np.abs(_np(got["out"]) - out) <= t_out)[:, hidden].all()
    assert (np.abs(_np(got["lse"]) - lse) <= t_lse)[:, hidden].all()
    # the last node's own row sees them: at head 1 its score is infinite or no number, at head 0 so is its value
    g = _np(got["out"])[:, rows - 1]
    assert np.isinf(g[:, :hq // 2, 11]).all()


@pytest.mark.parametrize("rows,hq", MANY)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_and_large_values_that_every_row_sees(sv, h, dtype, rows, hq):  # noqa: F811
    """An infinite value makes its column infinite; two of opposite sign make
    theirs NaN; a NaN is one; the largest finite value stays finite."""
    import torch

    c = Case(rows, dtype, 2, rows, hq, 2, 128, 16, [200, rows], "tree", q_scale=0.5)
    big = float(torch.finfo(c.dtype).max)
    for t, head, col, val in ((5, 0, 3, math.inf), (6, 0, 4, -math.inf), (5, 0, 5, math.inf), (6, 0, 5, -math.inf),
                              (2, 1, 7, math.nan), (1, 1, 9, big), (2, 1, 10, -big)):
        _set(c, c.vc_t, 0, t, head, col, val)
    got = c.call(sv, h)
    # (position 1 and 2 are in the first tile of any kernel: the maximum that weights are taken against is not below
    # their scores, so that weight * value stays below the type's largest)
    c.check(got)
    g = _np(got["out"])[0]
    half = hq // 2
    assert np.isposinf(g[:, :half, 3]).all() and np.isneginf(g[:, :half, 4]).all() and np.isnan(g[:, :half, 5]).all()
    assert np.isnan(g[:, half:, 7]).all() and (g[:, half:, 9] > 1e30).all() and (g[:, half:, 10] < -1e30).all()
    assert np.isnan(g).sum() == rows * hq and np.isinf(g).sum() == rows * hq


@pytest.mark.parametrize("rows,hq", MANY)
@pytest.mark.parametrize("key", ["lowest", "infinite"])
@pytest.mark.parametrize("query", [1.0, 5000.3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys_that_weigh_nothing(sv, h, dtype, query, key, rows, hq):  # noqa: F811
    """A prefix key whose score is below all range (as masks by the type's
    lowest value make them) has weight zero, and nothing else of the row
    changes, whatever finite value lies there."""
    import torch

    c = Case(rows + 7, dtype, 2, rows, hq, 2, 64, 16, [150, rows + 40], "tree")
    big = float(torch.finfo(c.dtype).max)
    c.kc_t[:, :, :, 7] = 0
    c.q_t[..., 7] = query
    c.q = _np(c.q_t)
    # the reference: the key's score 1e4 below the others, where float64 has no weight left; the bound's magnitudes are
    # those of the other keys, whose sums the kernels round
    out, lse, status, avg, _ = P.attention(c.q, *_flat(c, 5, -1e4), c.lens, c.parents, c.scale)
    mag = P.attention(c.q, *_flat(c, 5, 0.0), c.lens, c.parents, c.scale)[4]
    t_out, t_lse = P.attention_bounds(out, lse, avg, mag, int(c.lens.max()), 64, dtype == "bf16")
    for b in range(2):
        _set(c, c.kc_t, b, 5, slice(None), 7, -big if key == "lowest" else -math.inf)
        _set(c, c.vc_t, b, 5, slice(None), 3, big)
    got = c.call(sv, h)
    assert got["row_status"].tolist() == [0, 0]
    assert (np.abs(_np(got["out"]) - out) <= t_out).all()
    assert (np.abs(_np(got["lse"]) - lse) <= t_lse).all()


def _flat(c, t, key):
    """Keys, values and tables of a case in blocks of one position, where position t of each sequence has `key` in its
    column 7 (all others have 0 there) and values of 0."""
    kc, vc = _np(c.kc_t), _np(c.vc_t)
    k = np.ascontiguousarray(kc.transpose(0, 2, 1, 3)).reshape(-1, kc.shape[1], 1, kc.shape[3])
    v = np.ascontiguousarray(vc.transpose(0, 2, 1, 3)).reshape(-1, vc.shape[1], 1, vc.shape[3])
    tables = np.full((len(c.lens), int(c.lens.max())), -1, np.int64)
    for b, n in enumerate(c.lens):
        at = np.arange(int(n))
        tables[b, :n] = c.tables[b, at // 16].astype(np.int64) * 16 + at % 16
        k[tables[b, t]] = key * (np.arange(kc.shape[3]) == 7)
        v[tables[b, t]] = 0.0
    return k, v, tables


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,rows,rot,inter", [(3, 9, 64, False), (40, 50, 64, False), (40, 50, 32, True), (3, 9, 6, False)])
def test_append_leaves_padding_alone(sv, h, dtype, B, rows, rot, inter):  # noqa: F811
    """Whatever the rows behind a sequence's count hold, the cache and the
    queries are the same bits; padding's queries are zero."""
    import torch

    dt = _dtype(dtype)
    rng = np.random.default_rng(B)
    counts = rng.integers(0, rows + 1, size=B).astype(np.int32)
    lens = counts + rng.integers(0, 30, size=B).astype(np.int32) * (counts > 0)
    tables, blocks = _tables(rng, lens, 16)
    inv = _dev((10000.0 ** (-np.arange(rot // 2) * 2 / rot)).astype(np.float32))
    x, _ = _rounded(rng, (B, rows, 8, 64), dt)
    pad = torch.from_numpy(np.arange(rows)[None] >= counts[:, None]).cuda()
    results = []
    for fill in (0.0, math.nan, float(torch.finfo(dt).max), -math.inf):
        y = x.clone()
        y[pad] = fill
        kc, vc = (torch.zeros((blocks, 2, 16, 64), dtype=dt, device="cuda") for _ in range(2))
        got = sv.specv_cache_append(h, kc, vc, _dev(tables), _dev(lens.astype(np.int32)), y[:, :, 4:6], y[:, :, 6:],
                                    q=y[:, :, :4], inv_freq=inv, interleaved=inter, row_counts=_dev(counts))
        assert not got["row_status"].any() and not got["q_out"][pad].any()
        results.append((got["q_out"], kc, vc))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


@pytest.mark.parametrize("rows,hq", MANY)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_scale_of_zero_weighs_evenly(sv, h, dtype, rows, hq):  # noqa: F811
    """Whatever the scores' size: here 1e31."""
    c = Case(rows + 3, dtype, 2, rows, hq, 2, 64, 16, [90, rows + 5], "tree", q_scale=1e30)
    c.check(c.call(sv, h, scale=0.0), scale=0.0)
    c.check(c.call(sv, h, scale=-0.0), scale=0.0)


def test_scales_out_of_range_are_refused(sv, h):  # noqa: F811
    """A scale has to be finite, and so has scale * log2(e), the factor of the
    scores in base 2."""
    c = Case(1, "f32", 1, 2, 2, 2, 64, 16, [20], "tree", q_scale=1e-30)
    before = sv.specv_launch_count(h)
    for scale in (3e38, -2.4e38, math.inf, -math.inf, math.nan, 1e40):
        with pytest.raises(sv.SpecvError):
            c.call(sv, h, scale=scale)
    assert sv.specv_launch_count(h) == before
    got = c.call(sv, h, scale=2.3e38)
    assert np.isfinite(_np(got["out"])).all() and np.isfinite(_np(got["lse"])).all()
    c.check(c.call(sv, h, scale=1e-45), scale=1e-45)
