"""The calls on the paged KV cache at shapes between their kernels' tiles:
many query heads to a kv head, row tiles without rows, long prompts, blocks
that sequences share."""
import numpy as np
import pytest

import cache_plain as P
from test_gpu_cache import Case, _dev, _np, _rounded, h, sv, test_append_matches_the_formula  # noqa: F401

pytestmark = pytest.mark.gpu
check_append = test_append_matches_the_formula
del test_append_matches_the_formula

GROUPS = [
    # B, rows, q heads, kv heads, dim, block, lengths, tree
    (2, 32, 16, 1, 128, 16, [32, 300], "tree"),   # 512 rows a kv head: two row tiles of 256, queries as boxes of 8 rows
    (1, 32, 32, 1, 64, 16, [200], "tree"),        # 1024 rows, boxes of 4
    (2, 9, 32, 1, 128, 16, [9, 300], "tree"),     # 288 rows: the last tile's second half has none
    (2, 5, 32, 1, 64, 32, [5, 140], "star"),      # 160 rows: 32 in the second half
    (2, 17, 16, 2, 128, 16, [40, 290], "tree"),   # 136 rows: 8 in the second half
    (2, 16, 16, 2, 128, 16, [16, 290], "line"),   # 256 rows: both halves full
    (2, 8, 16, 1, 128, 16, [8, 129], "tree"),     # 128 rows: one half
    (2, 12, 24, 2, 112, 64, [12, 200], "tree"),   # 144 rows, groups that fill no row tile
    (1, 32, 128, 1, 128, 16, [180], "tree"),      # a row a box, 4096 rows
    (1, 3, 256, 1, 64, 16, [150], "tree"),        # groups above a row tile
    (1, 1, 256, 1, 128, 16, [300], "chain"),
    (2, 2, 64, 1, 16, 128, [2, 260], "tree"),
    (3, 32, 16, 2, 80, 8, [33, 127, 128], "star"),
    (3, 25, 32, 4, 64, 256, [25, 256, 513], "tree"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", GROUPS, ids=lambda s: "B%d_R%d_H%d-%d_D%d_bs%d_%s" % (s[:6] + (s[7],)))
def test_many_query_heads_to_a_kv_head(sv, h, dtype, shape):  # noqa: F811
    B, rows, hq, hkv, dim, bs, lens, kind = shape
    c = Case(B * 900 + rows * 10 + dim, dtype, B, rows, hq, hkv, dim, bs, lens, kind)
    c.check(c.call(sv, h))


@pytest.mark.parametrize("rows,hq", [(3, 4), (17, 8), (32, 16)])
def test_sequences_that_share_blocks(sv, h, rows, hq):  # noqa: F811
    """A common prefix held once: block tables that name the same blocks."""
    c = Case(rows, "bf16", 4, rows, hq, 2, 64, 16, [rows + 200, rows + 230, rows + 64, rows + 300], "tree", poison=False)
    c.tables[1, :12], c.tables[2, :4], c.tables[3, :12] = c.tables[0, :12], c.tables[0, :4], c.tables[0, :12]
    c.check(c.call(sv, h))


PROMPTS = [
    # B, rows, q heads, kv heads, dim, block, lengths, tree, rot, interleaved, counts
    (2, 2500, 2, 1, 64, 16, [2600, 1999], "chain", 64, False, [2500, 1999]),
    (1, 3500, 1, 1, 16, 1, [3501], "chain", 8, True, None),
    (2, 2100, 3, 1, 32, 64, [0, 2100], "chain", 6, False, [0, 2100]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", PROMPTS, ids=lambda s: "B%d_R%d_H%d-%d_D%d_bs%d" % s[:6])
def test_long_prompts(sv, h, dtype, shape):  # noqa: F811
    check_append(sv, h, dtype, shape)


@pytest.mark.parametrize("rows,hq", [(3, 4), (17, 8), (32, 16)])
def test_append_then_attention_for_each_count(sv, h, rows, hq):  # noqa: F811
    """A batch whose passes differ in rows, as the header has it: appended with
    row counts, attended to by a call for each count."""
    import torch

    rng = np.random.default_rng(rows)
    c = Case(rows, "f32", 4, rows, hq, 2, 64, 16, [rows + 40] * 4, "tree", poison=False)
    counts = np.array([rows, 1 + rows // 2, rows, 1 + rows // 2], np.int32)
    lens = 40 + counts
    (k_t, k), (v_t, v) = (_rounded(rng, (4, rows, 2, 64), c.dtype) for _ in range(2))
    tables, par = _dev(c.tables), _dev(c.parents)
    kc, vc = c.kc.copy(), c.vc.copy()
    got = sv.specv_cache_append(h, c.kc_t, c.vc_t, tables, _dev(lens), k_t, v_t, parents=par, row_counts=_dev(counts))
    assert not got["row_status"].any()
    P.append(kc, vc, c.tables, lens, k, v, parents=c.parents, counts=counts)
    np.testing.assert_array_equal(_np(c.kc_t), kc)
    for n in sorted(set(counts.tolist())):
        pick = np.flatnonzero(counts == n)
        at = torch.from_numpy(pick).cuda()
        sub_par = c.parents[pick][:, :n - 1]
        one = sv.specv_tree_attention(h, c.q_t[at][:, :n].contiguous(), c.kc_t, c.vc_t, tables[at].contiguous(),
                                      _dev(lens[pick]), parents=_dev(sub_par), lse=True)
        out, lse, status, avg, mag = P.attention(c.q[pick][:, :n], kc, vc, c.tables[pick], lens[pick], sub_par, c.scale)
        t_out, t_lse = P.attention_bounds(out, lse, avg, mag, int(lens.max()), 64, False)
        assert not one["row_status"].any() and not status.any()
        assert (np.abs(_np(one["out"]) - out) <= t_out).all() and (np.abs(_np(one["lse"]) - lse) <= t_lse).all()


def test_workspace_of_invalid_sizes_is_none(sv, h):  # noqa: F811
    """0 where specv_tree_attention refuses the sizes, at every end of them."""
    need = lambda dt=sv.SPECV_BF16, kv=8, dim=128, q=32, batch=4, rows=17: (  # noqa: E731
        sv.specv_tree_attention_workspace(h, dt, kv, dim, q, batch, rows))
    assert need() > 0 and need(kv=65536, q=65536) > 0 and need(kv=1, q=65536, rows=32) > 0
    for kw in (dict(dt=2), dict(kv=0), dict(dim=8), dict(dim=24), dict(dim=272), dict(q=0), dict(q=33),
               dict(kv=1, q=65537), dict(kv=1, q=2 ** 30, rows=32), dict(kv=131072, q=131072), dict(batch=0),
               dict(batch=513), dict(rows=0), dict(rows=33)):
        assert need(**kw) == 0, kw


@pytest.mark.parametrize("rows,hq", [(1, 4), (3, 4), (17, 8), (32, 16)])
def test_tables_and_lengths_written_just_before(sv, h, rows, hq):  # noqa: F811
    """Kernels that write the tables, lengths, trees and queries, with the
    call right behind them, many times over: every call sees its own."""
    import torch

    cases = [Case(rows + i, "bf16", 3, rows, hq, 2, 64, 16, lens, "tree", width=40, poison=False)
             for i, lens in enumerate(([rows, 500, 90], [610, rows + 1, 33 + rows]))]
    blocks = max(c.kc_t.shape[0] for c in cases)
    kc = torch.zeros((2, blocks, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    src = []
    for i, c in enumerate(cases):
        kc[i, :c.kc_t.shape[0]], vc[i, :c.vc_t.shape[0]] = c.kc_t, c.vc_t
        shift = np.where(c.tables >= 0, c.tables + i * blocks, -1).astype(np.int32)  # in one pool of both
        src.append((_dev(shift), _dev(c.lens), _dev(c.parents), c.q_t))
    pool_k, pool_v = kc.view(-1, 2, 16, 64), vc.view(-1, 2, 16, 64)
    now = [torch.zeros_like(t) for t in src[0]]
    outs = []
    for i in range(40):
        for t, s in zip(now, src[i % 2]):
            t.copy_(s)
        outs.append(sv.specv_tree_attention(h, now[3], pool_k, pool_v, now[0], now[1], parents=now[2], lse=True))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        if i < 2:
            cases[i].check(out)
        else:
            assert torch.equal(out["out"], outs[i % 2]["out"]) and torch.equal(out["lse"], outs[i % 2]["lse"])
