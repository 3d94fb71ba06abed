"""Pins of the plain restatements that the cache kernels are checked with,
and the refusals of the cache calls that need no device."""
import ctypes

import numpy as np
import pytest

import cache_plain as P


def test_page_tree_depths_and_ancestors():
    """The page's six-node tree (s.3): depths 0,1,1,2,2,2 below the prefix's
    last token, which is row 0 here, one level up."""
    ok, depth, seen = P.tree([-1, 0, 0, 1, 1, 2], 7)
    assert ok and depth == [0, 1, 2, 2, 3, 3, 3]
    assert [sorted(s) for s in seen] == [[0], [0, 1], [0, 1, 2], [0, 1, 3], [0, 1, 2, 4], [0, 1, 2, 5], [0, 1, 3, 6]]
    assert P.tree([0], 2)[0] is False and P.tree([-2], 2)[0] is False


def test_rotation_keeps_relative_positions():
    """Products of rotated vectors depend on the difference of positions only."""
    rng = np.random.default_rng(0)
    f = 10000.0 ** (-np.arange(8) / 8)
    a, b = rng.normal(size=(1, 16)), rng.normal(size=(1, 16))
    for inter in (False, True):
        one = np.sum(P.rotate(a, 7, f, inter) * P.rotate(b, 3, f, inter))
        two = np.sum(P.rotate(a, 1007, f, inter) * P.rotate(b, 1003, f, inter))
        assert abs(one - two) < 1e-10
        assert np.allclose(P.rotate(a, 0, f, inter), a)


def test_attention_of_a_chain_is_causal_attention():
    rng = np.random.default_rng(1)
    q, kc, vc = rng.normal(size=(1, 3, 2, 16)), rng.normal(size=(4, 1, 4, 16)), rng.normal(size=(4, 1, 4, 16))
    tables = np.array([[2, 0, 3]], np.int32)
    out, lse, st, _, _ = P.attention(q, kc, vc, tables, [9], None, 0.25)
    K, V = kc[[2, 0, 3], 0].reshape(12, 16), vc[[2, 0, 3], 0].reshape(12, 16)
    for r in range(3):
        s = q[0, r] @ K[:7 + r].T * 0.25
        e = np.exp(s)
        assert np.allclose(out[0, r], e @ V[:7 + r] / e.sum(1, keepdims=True))
        assert np.allclose(lse[0, r], np.log(e.sum(1)))
    assert st[0] == 0
    star = P.attention(q, kc, vc, tables, [9], np.array([[-1, -1]]), 0.25)[0]
    assert not np.allclose(star[0, 2], out[0, 2]) and np.allclose(star[0, 1], out[0, 1])


def test_compaction_in_order_of_the_path():
    kc = np.arange(12.0).reshape(1, 3, 1, 4, 1)
    vc = -kc
    tables = np.array([[1, 2, 0]], np.int32)
    st = P.compact(kc, vc, tables, [10], np.array([[1, 2, 4, -1, -1]]), [3])
    # nodes at positions 5..9: blocks 2, 2, 2, 0, 0
    assert st[0] == 0
    flat = kc[0, [1, 2, 0], 0].reshape(-1)
    assert flat[5:10].tolist() == [10, 11, 1, 0, 1]
    assert np.array_equal(vc, -kc)


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_57_gb300 import _lib, build

    build.build()
    return _lib.load()


def test_null_handle_is_refused_without_a_device(lib):
    from speculative_decoding_verification_57_gb300 import _lib

    c = _lib.SpecvKvCache()
    assert lib.specv_cache_append(None, ctypes.byref(c), None, 0, 0, None, 0, None, 0, None, 0, 0, None, None, 1, 1,
                                  None, None, None) == 1
    assert lib.specv_tree_attention(None, ctypes.byref(c), None, 0, 1, None, 1, 1, 1.0, None, None, None, None, 0,
                                    None) == 1
    assert lib.specv_cache_compact(None, ctypes.byref(c), 1, 0, None, None, 1, 1, None, None) == 1
    assert lib.specv_tree_attention_workspace(None, 1, 8, 128, 32, 1, 1) == 0


def test_binding_refuses_host_tensors_and_types():
    import torch

    import speculative_decoding_verification_57_gb300 as sv

    h = sv.Handle(None, 0, 4, 4, 100)
    pool = torch.zeros((2, 1, 4, 16), dtype=torch.bfloat16)
    one = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="handle's device"):
        sv.specv_tree_attention(h, pool, pool, pool, one, one[0])
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        sv.specv_cache_compact(h, pool.half(), pool.half(), one, one[0], one, one[0])
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        sv.specv_cache_append(h, None, None, one, one[0], pool, pool)
