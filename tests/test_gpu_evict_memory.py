"""Eviction: memory that it writes may not be memory that it reads, and
lengths as far as they are counted."""
import pytest

from test_gpu_cache import h, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["seq_lens", "evicted", "row_status"])
def test_eviction_refuses_outputs_in_its_inputs(sv, h, name):  # noqa: F811
    import torch

    i32 = dict(dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((4, 2, 16, 64), device="cuda") for _ in range(2))
    both = torch.zeros(12, **i32)  # tables of 3 x 2, lengths, and what lies beside them
    tables, lens = both[:6].view(3, 2), both[6:9]
    mass = torch.zeros((3, 2, 32), device="cuda")
    before = sv.specv_launch_count(h)
    for at in (lens, both[5:8], both[7:10], both[0:3], both[4:7]):
        with pytest.raises(sv.SpecvError):
            sv.specv_cache_evict(h, kc, vc, tables, lens, mass, 4, out={name: at})
    assert sv.specv_launch_count(h) == before
    got = sv.specv_cache_evict(h, kc, vc, tables, lens, mass, 4, out={name: both[9:12]})  # beside them is fine
    assert sv.specv_launch_count(h) == before + 1 and not got["row_status"].any()


def test_eviction_at_the_longest_lengths(sv, h):  # noqa: F811
    """Nothing to move at 2^31 - 4096 positions; lengths beyond that are refused, as counters of positions
    would leave their type."""
    import torch

    i32 = dict(dtype=torch.int32, device="cuda")
    most, width = 2 ** 31 - 4096, 2 ** 31 - 1
    kc = torch.zeros((1, 1, 65536, 256), dtype=torch.bfloat16, device="cuda")
    tables = torch.zeros((1, 32768), **i32)
    mass = torch.ones((1, 1, width), device="cuda")
    out = torch.zeros_like(mass)
    for n in (most + 1, 2 ** 31 - 513, 2 ** 31 - 512, 2 ** 31 - 1):
        for budget in (10, width):
            got = sv.specv_cache_evict(h, kc, kc, tables, torch.tensor([n], **i32), mass, budget, out={"mass": out})
            assert got["row_status"].tolist() == [sv.ST_LENGTH] and got["seq_lens"].tolist() == [n]
            assert got["evicted"].tolist() == [0]
    assert out[0, 0, ::65536].sum() == 0
    got = sv.specv_cache_evict(h, kc, kc, tables, torch.tensor([most], **i32), mass, width, out={"mass": out})
    assert got["row_status"].tolist() == [0] and got["seq_lens"].tolist() == [most]
    assert bool((out[0, 0, :2 ** 30] == 1).all()) and bool((out[0, 0, 2 ** 30:most] == 1).all())
    assert bool((out[0, 0, most:] == 0).all())
