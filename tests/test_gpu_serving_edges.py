"""The serving calls on both sides of the sizes at which another kernel, or
another number of threads, takes over."""
import numpy as np
import pytest

import cache_plain as P
import serving_plain as S
from test_gpu_cache import BF16_HALF, F32_HALF, _dev, _dtype, _np, _rounded, _tables, h, sv  # noqa: F401
from test_gpu_prefix import Shared, _exact_rows
from test_gpu_serving import _mass_case, _mass_check, _norm_call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("a_sm", [3, 5])
@pytest.mark.parametrize("past", [0, 1])
@pytest.mark.parametrize("trees", [False, True])
def test_append_norm_where_threads_change(sv, h, dtype, a_sm, past, trees):  # noqa: F811
    """As many tokens as the SMs hold at three or five each, and one more: a prompt, or trees of four."""
    import torch

    tokens = torch.cuda.get_device_properties(0).multi_processor_count * a_sm + past
    if trees:
        B, rows, kind, lens = tokens // 4 + past, 4, "tree", [4 + i % 7 for i in range(tokens // 4 + past)]
    else:
        B, rows, kind, lens = 1, tokens, "chain", [tokens + 9]
    shape = (B, rows, 6, 2, 64, 16, lens, kind, 64, False, None, 0, True)
    call, pools, ref, ref_k, ref_v = _norm_call(sv, h, _dtype(dtype), shape, (True, True))
    (kc_t, kc), (vc_t, _) = pools
    got = call(kc_t, vc_t)
    q_out, status, written, (q_mag, k_mag) = ref
    half = BF16_HALF if dtype == "bf16" else F32_HALF
    np.testing.assert_array_equal(got["row_status"].cpu().numpy(), status)
    np.testing.assert_array_equal(_np(vc_t), ref_v)
    assert (np.abs(_np(kc_t) - ref_k) <= S.append_norm_bound(ref_k, k_mag, 64, half)).all()
    assert (np.abs(_np(got["q_out"]) - q_out) <= S.append_norm_bound(q_out, q_mag, 64, half)).all()


@pytest.mark.parametrize("masses", ["spread", "ties", "late", "early"])
@pytest.mark.parametrize("n,budget,recent,first", [(70000, 30000, 100, 4), (131072, 20480, 3000, 0), (40000, 39000, 1, 64),
                                                   (5000, 2300, 200, 7)])
def test_eviction_with_many_lists_of_moves(sv, h, n, budget, recent, first, masses):  # noqa: F811
    """Lists of 1024 moves, each found where the last one ended: holes and kept positions spread, all of
    them together at the ends, and ties that a list's end cuts."""
    import torch

    rng = np.random.default_rng(n)
    lens = np.array([n, n - 300], np.int32)
    tables, blocks = _tables(rng, lens, 64)
    pools = [_rounded(rng, (1, blocks, 2, 64, 16), torch.bfloat16) for _ in range(2)]
    m = rng.exponential(size=(1, 2, 2, n)).astype(np.float32)
    if masses == "ties":
        m = np.floor(m * 3)
    if masses == "late":
        m = np.sort(m, -1)
    if masses == "early":
        m = -np.sort(-m, -1)
        m[0, 0, 0, ::5] = 0
    ref = [p[1].copy() for p in pools]
    places, new, status = S.evict(*ref, tables, lens, m, budget, recent, first)
    got = sv.specv_cache_evict(h, pools[0][0][0], pools[1][0][0], _dev(tables), _dev(lens), _dev(m[0]), budget, recent=recent,
                               first=first)
    torch.cuda.synchronize()
    assert got["row_status"].tolist() == [0, 0] and got["seq_lens"].tolist() == new.tolist()
    for p, r in zip(pools, ref):
        np.testing.assert_array_equal(_np(p[0]), r)
    g = got["mass"].cpu().numpy()
    for b in range(2):
        for hh in range(2):
            place = places[0][b][hh]
            np.testing.assert_array_equal(g[b, hh, :len(place) if place is not None else lens[b]],
                                          m[0, b, hh, place] if place is not None else m[0, b, hh, :lens[b]])


@pytest.mark.parametrize("dim", [64, 128, 112])
@pytest.mark.parametrize("B,rows,hq", [
    (16, 1, 1), (17, 1, 1),    # a kv head's rows of the batch on mma.sync, and on tcgen05
    (32, 4, 1), (43, 3, 1),    # one row tile, and two side by side
    (32, 32, 1), (41, 25, 1),  # eight row tiles side by side, and tiles of 256
])
def test_prefix_attention_where_kernels_change(sv, h, B, rows, hq, dim):  # noqa: F811
    c = Shared(B + rows + dim, "bf16", B, rows, hq, 1, dim, 16, 4096, [rows + (37 * i) % 200 for i in range(B)])
    got = c.call(sv, h)
    out, lse, avg, mag = _exact_rows(c)
    assert not got["row_status"].any()
    t_out, t_lse = P.attention_bounds(out, lse, avg, mag, int(c.lens.max()), dim, True)
    assert (np.abs(_np(got["out"]) - out) <= t_out).all()
    assert (np.abs(_np(got["lse"]) - lse) <= t_lse).all()
    again = c.call(sv, h)
    assert (got["out"] == again["out"]).all() and (got["lse"] == again["lse"]).all()


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 128), ("bf16", 144), ("f32", 64)])
@pytest.mark.parametrize("rows,group", [(8, 1), (9, 1), (32, 1), (11, 3), (16, 5), (27, 3), (32, 4), (3, 43), (32, 8), (1, 257)])
def test_mass_where_kernels_change(sv, h, dtype, dim, rows, group):  # noqa: F811
    """Queries of a kv head on both sides of a tile of eight, of four and ten tiles, of two sets of
    queries and of tcgen05's one."""
    import torch

    c = _mass_case(rows + group, dtype, (2, rows, 2 * group, 2, dim, 16, [rows + 150, rows], "tree", 5))
    got = sv.specv_attention_mass(h, c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), _dev(c.lse), first=5,
                                  parents=None if c.parents is None else _dev(c.parents))
    torch.cuda.synchronize()
    _mass_check(c, got, None, 5, c.lse, 0.0)
