"""Pins of the plain restatements in serving_plain.py: closed forms and small
examples worked out by hand."""
import numpy as np

import cache_plain as P
import serving_plain as S


def test_norm_of_equal_values_is_the_weight():
    w = np.arange(4.0)
    np.testing.assert_allclose(S.norm(np.full((2, 4), -3.0), w, 0.0, 1.0), -np.tile(w + 1, (2, 1)))
    x = np.array([[3.0, 4.0]])
    np.testing.assert_allclose(S.norm(x, np.ones(2), 0.0, 0.0), x / np.sqrt(12.5))
    np.testing.assert_allclose(S.norm(x, np.ones(2), 12.5, 0.0), x / 5.0)
    assert S.norm(x, None, 1.0, 1.0) is not x and (S.norm(x, None, 1.0, 1.0) == x).all()


def test_append_without_norms_is_the_plain_append():
    rng = np.random.default_rng(1)
    tables, lens = np.array([[2, 0], [1, 3]]), np.array([5, 7])
    k, v, q = rng.normal(size=(2, 3, 2, 8)), rng.normal(size=(2, 3, 2, 8)), rng.normal(size=(2, 3, 4, 8))
    inv, par = np.array([1.0, 0.1, 0.01]), np.array([[-1, -1], [-1, 0]])
    for inter in (False, True):
        one, two = [np.zeros((2, 4, 2, 4, 8)) for _ in range(2)]
        a = P.append(*one, tables, lens, k, v, q=q, inv_freq=inv, interleaved=inter, parents=par)
        b = S.append_norm(*two, tables, lens, k, v, q=q, inv_freq=inv, interleaved=inter, parents=par)
        np.testing.assert_allclose(one, two)
        np.testing.assert_allclose(a[0], b[0])
        # one axis with the same positions, or positions behind by an offset, are the same again
        depth = np.array([[0, 1, 1], [0, 1, 2]]) + (lens - 3)[:, None]
        c = S.append_norm(*two, tables, lens, k, v, q=q, inv_freq=inv, interleaved=inter, positions=depth[:, :, None])
        np.testing.assert_allclose(a[0], c[0])
        d = S.append_norm(*two, tables, lens, k, v, q=q, inv_freq=inv, interleaved=inter, parents=par,
                          offsets=np.array([0, 9]))
        np.testing.assert_allclose(a[0][0], d[0][0])
        assert not np.allclose(a[0][1], d[0][1])


def test_axes_turn_their_own_pairs():
    x = np.array([[1.0, 1.0, 0.0, 0.0]])
    k = np.tile(x, (1, 1, 1, 1))
    kc = np.zeros((1, 1, 1, 4))
    S.append_norm(kc, kc.copy(), np.array([[0]]), np.array([1]), k, k, inv_freq=np.array([np.pi / 2, np.pi / 2]),
                  positions=np.array([[[1, 2]]]), axis=[0, 1])
    np.testing.assert_allclose(kc[0, 0, 0], [0, -1, 1, 0], atol=1e-15)


def test_attention_of_a_shared_prefix_is_attention_over_the_whole():
    rng = np.random.default_rng(2)
    kc, vc = rng.normal(size=(9, 2, 4, 8)), rng.normal(size=(9, 2, 4, 8))
    q = rng.normal(size=(3, 2, 4, 8))
    tables = np.array([[7, 1, 2, -1], [7, 1, 3, 4], [7, 1, -1, -1]])
    lens = np.array([11, 14, 0])
    a = P.attention(q, kc, vc, tables, lens, None, 0.3)
    other = tables.copy()
    other[:, :2] = 99  # what the sequences' own tables say of the prefix is not looked at
    b = S.prefix_attention(q, kc, vc, other, lens, np.array([7, 1]), 8, None, 0.3)
    for x, y in zip(a, b):
        np.testing.assert_array_equal(x, y)
    status = S.prefix_attention(q, kc, vc, tables, np.array([9, 17, 0]), np.array([7, 1]), 8, None, 0.3)[2]
    assert status.tolist() == [2048, 2048, 0]
    assert S.prefix_attention(q, kc, vc, tables, lens, np.array([7, 9]), 8, None, 0.3)[2].tolist() == [4096, 4096, 0]
    assert S.prefix_attention(q, kc, vc, tables, lens, np.array([7, 1]), 6, None, 0.3)[2].tolist() == [2048, 2048, 0]


def test_masses_of_a_row_add_up_to_one():
    rng = np.random.default_rng(3)
    kc, vc = rng.normal(size=(6, 2, 4, 8)), rng.normal(size=(6, 2, 4, 8))
    q = rng.normal(size=(2, 3, 4, 8))
    tables, lens, par = np.array([[5, 1, 2], [0, 3, 4]]), np.array([9, 12]), np.array([[-1, -1], [-1, 0]])
    _, lse, _, _, _ = P.attention(q, kc, vc, tables, lens, par, 0.5)
    got, status, written, _ = S.mass(q, kc, tables, lens, lse, par, 0.5, None, 0, 12)
    assert not status.any() and written[0, :, :9].all() and not written[0, :, 9:].any()
    np.testing.assert_allclose(got.sum(-1), 3 * 2)  # three rows, two query heads
    lse[0, 1] = np.inf
    got, _, _, _ = S.mass(q, kc, tables, lens, lse, par, 0.5, np.ones((2, 2, 12)), 4, 12)
    np.testing.assert_allclose(got[0].sum(-1) - 6, [x for x in S.mass(q, kc, tables, lens, lse, par, 0.5, None, 4, 12)[0][0].sum(-1)])


def test_eviction_by_hand():
    c = np.arange(12.0).reshape(1, 3, 1, 4, 1).copy()  # positions 0..11 in blocks 0, 1, 2
    tables, m = np.array([[0, 1, 2]]), np.zeros((1, 1, 1, 12))
    #            0  1  2  3  4  5  6  7  8  9 | 10 11 recent
    m[0, 0, 0] = [9, 1, 5, 0, 5, 8, 2, 5, 3, 7, 0, 0]
    places, new, status = S.evict(c, c.copy(), tables, np.array([12]), m, 7, 2, 1)
    # four of positions 1..9 stay: 5, 9, then 2 and 4 of the three fives; holes 1 and 3 take 5 and 9
    assert places[0][0][0] == [0, 5, 2, 9, 4, 10, 11] and new.tolist() == [7] and status.tolist() == [0]
    assert c.reshape(-1)[:7].tolist() == [0, 5, 2, 9, 4, 10, 11]
    assert S.evict(c, c.copy(), tables, np.array([7]), m, 7, 2, 1)[0][0][0][0] is None
