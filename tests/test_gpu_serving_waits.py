"""The bounded waits of the tcgen05 kernels of gathered weight and of the
sequences' part behind a shared prefix: a copy that never arrives is told for
every sequence that its CTA's run touches, and for no other, whatever the
status held before."""
import numpy as np
import pytest

from test_gpu_cache import Case, _dev, sv  # noqa: F401  (sv is a fixture)
from test_gpu_prefix import Shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [16, 5])  # boxes, and 16-byte copies
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,hq", [(3, 8), (32, 16)])  # two sets of queries, and one
def test_a_missing_copy_of_the_gathered_weight_is_told(sv, bs, dim, rows, hq):  # noqa: F811
    """400 sequences of a tile for each of two kv heads: the run of CTA 0 holds some of
    them from their start, and most of these come behind the wait that runs out."""
    import torch

    handle = sv.specv_create(0, max_batch=512, max_k=31, vocab=1000)
    B = 400
    c = Case(rows + dim + bs, "bf16", B, rows, hq, 2, dim, bs, [40 + i % 80 for i in range(B)], "tree", poison=False)
    lse = c.call(sv, handle)["lse"]
    args = (c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), lse)

    def call():
        out = {"mass": torch.full((B, 2, c.tables.shape[1] * bs), -7.0, device="cuda"),
               "row_status": torch.full((B,), -1, dtype=torch.int32, device="cuda")}
        got = sv.specv_attention_mass(handle, *args, parents=_dev(c.parents), out=out)
        torch.cuda.synchronize()
        return got["mass"], got["row_status"].cpu().numpy()

    want, status = call()
    assert not status.any()
    for use in (0, 1, 2, 4):
        sv.specv_test_withhold_stage(handle, use, 2000)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        mass, status = call()
        end.record()
        end.synchronize()
        n = int(np.count_nonzero(status))  # one run: the first sequences
        assert 3 <= n < 20 and (status[:n] == sv.ST_TIMEOUT).all() and not status[n:].any(), (use, status[:20])
        assert torch.equal(mass[n:], want[n:]), use
        assert start.elapsed_time(end) < 150, use  # no role waits for what is over (2000 polls take less than 10 ms)
        mass, status = call()
        assert not status.any() and torch.equal(mass, want), use
    sv.specv_destroy(handle)


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,hq,prefix,B", [(17, 8, 160, 120), (17, 8, 12000, 40), (32, 16, 160, 120), (17, 8, 30000, 14)])
def test_a_missing_copy_of_the_sequences_part_is_told(sv, bs, dim, rows, hq, prefix, B):  # noqa: F811
    """Sequences of two to four tiles for each of two kv heads behind a short prefix,
    beside a long one (two tiles a sequence and head, more of the prefix), and so few that they go the way of
    row tiles side by side: those that CTA 0's run of the sequences' launch touches are told, the others are the same bits."""
    import torch

    handle = sv.specv_create(0, max_batch=512, max_k=31, vocab=1000)
    prefix = prefix // bs * bs
    c = Shared(rows + dim + bs, "bf16", B, rows, hq, 2, dim, bs, prefix, [150 + 7 * (i % 40) for i in range(B)])

    def call():
        out = {"row_status": torch.full((B,), -1, dtype=torch.int32, device="cuda")}
        got = c.call(sv, handle, out=out)
        return got, got["row_status"].cpu().numpy()

    want, status = call()
    assert not status.any()
    for use in (0, 1, 2, 3) if B > 14 else (0, 1):  # (two tiles a run, or one)
        sv.specv_test_withhold_stage(handle, 2 ** 20 + use, 2000)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        got, status = call()
        end.record()
        end.synchronize()
        n = int(np.count_nonzero(status))  # one run: the first sequences
        assert 1 <= n < B // 2 and (status[:n] == sv.ST_TIMEOUT).all() and not status[n:].any(), (use, status)
        for key in ("out", "lse"):
            assert torch.equal(got[key][n:], want[key][n:]), use
        assert start.elapsed_time(end) < 150, use
        again, status = call()
        assert not status.any(), use
        for key in ("out", "lse"):
            assert torch.equal(again[key], want[key]), use
    sv.specv_destroy(handle)


@pytest.mark.parametrize("dim,rows", [(128, 17), (128, 1), (64, 17)])
def test_no_call_of_the_gathered_weight_stands_still(sv, dim, rows):  # noqa: F811
    """Many calls over several sets of inputs: none takes the time of a wait that runs out (200 ms; a hundred calls take
    some 10), and all of them give the same bits."""
    import torch

    handle = sv.specv_create(0, max_batch=64, max_k=31, vocab=1000)
    sets = []
    for i in range(3):
        c = Case(i, "bf16", 64, rows, 32, 8, dim, 16, [1500 + (977 * (i + j)) % 1500 for j in range(64)], "tree", poison=False)
        q, kc, vc, tables, lens, par = c.q_t, c.kc_t, c.vc_t, _dev(c.tables), _dev(c.lens), _dev(c.parents)
        lse = sv.specv_tree_attention(handle, q, kc, vc, tables, lens, parents=par, lse=True)["lse"]
        out = {"mass": torch.zeros((64, 8, c.tables.shape[1] * 16), device="cuda"),
               "row_status": torch.zeros(64, dtype=torch.int32, device="cuda")}
        sets.append(((handle, q, kc, vc, tables, lens, lse), dict(parents=par, out=out)))
    first = [sv.specv_attention_mass(*a, **kw)["mass"].clone() for a, kw in sets]
    events = [torch.cuda.Event(enable_timing=True) for _ in range(151)]
    events[0].record()
    for e in events[1:]:
        for i in range(100):
            a, kw = sets[i % 3]
            sv.specv_attention_mass(*a, **kw)
        e.record()
    torch.cuda.synchronize()
    assert max(x.elapsed_time(y) for x, y in zip(events, events[1:])) < 100
    for want, (_, kw) in zip(first, sets):
        assert torch.equal(kw["out"]["mass"], want) and not kw["out"]["row_status"].any()
    sv.specv_destroy(handle)
