"""The bounded waits of tree attention's tcgen05 kernel: a copy that never
arrives, at every place of a run, is told for every sequence it touches."""
import pytest

from test_gpu_cache import Case, sv  # noqa: F401  (sv is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,hq", [(17, 8), (32, 16)])
def test_whatever_a_missing_copy_changes_is_told(sv, bs, dim, rows, hq):  # noqa: F811
    """Runs of eight tiles, sixteen slot uses (7 sequences of some 11,000
    positions, two kv heads: about 1230 tiles for 152 CTAs): the sequences
    whose results differ all have bit 64, the others are the same bits."""
    import torch

    handle = sv.specv_create(0, max_batch=64, max_k=31, vocab=1000)
    c = Case(rows + dim, "bf16", 7, rows, hq, 2, dim, bs, [11000 + 37 * i for i in range(7)], "tree", poison=False)
    want = c.call(sv, handle)
    assert not want["row_status"].any()
    for use in (0, 1, 2, 4, 5, 6, 7, 9, 10, 11, 12, 13):
        sv.specv_test_withhold_stage(handle, use, 20_000)
        got = c.call(sv, handle)
        late = (got["row_status"] & sv.ST_TIMEOUT) != 0
        assert late[0] and late.sum() < 7 and not (got["row_status"] & ~sv.ST_TIMEOUT).any(), use
        for key in ("out", "lse"):
            assert torch.equal(got[key][~late], want[key][~late]), use
    again = c.call(sv, handle)
    assert not again["row_status"].any()
    for key in ("out", "lse"):
        assert torch.equal(again[key], want[key])
    sv.specv_destroy(handle)


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("rows,hq", [(17, 8), (32, 16)])
def test_a_missing_copy_costs_its_own_waits_only(sv, bs, dim, rows, hq):  # noqa: F811
    """No role of a call that ran out waits for something that is over already
    (such a wait would run for 200 ms; 2000 polls take less than 10)."""
    import torch

    handle = sv.specv_create(0, max_batch=64, max_k=31, vocab=1000)
    c = Case(rows + dim, "bf16", 7, rows, hq, 2, dim, bs, [11000 + 37 * i for i in range(7)], "tree", poison=False)
    c.call(sv, handle)
    for use in (0, 1, 2, 3, 7):
        sv.specv_test_withhold_stage(handle, use, 2000)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        got = c.call(sv, handle)
        end.record()
        torch.cuda.synchronize()
        assert got["row_status"].tolist()[0] == sv.ST_TIMEOUT
        assert start.elapsed_time(end) < 150, use
    sv.specv_destroy(handle)
