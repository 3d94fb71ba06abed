"""Eviction: memory that it writes may not be memory that it reads."""
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
