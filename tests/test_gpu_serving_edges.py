"""The serving calls on both sides of the sizes at which another kernel, or
another number of threads, takes over."""
import numpy as np
import pytest

import serving_plain as S
from test_gpu_cache import BF16_HALF, F32_HALF, _dtype, _np, h, sv  # noqa: F401
from test_gpu_serving import _norm_call

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
