"""Norms of heads near the ends of fp32: sums of squares beyond the type, and
squares that vanish in it."""
import numpy as np
import pytest

import serving_plain as S
from test_gpu_cache import BF16_HALF, F32_HALF, _dev, _dtype, _np, h, sv  # noqa: F401

pytestmark = pytest.mark.gpu

# magnitudes of a head's values, as exponents: all, or the first alone
ENDS = [0, 61, 63.5, 64, 100, 126, 127, -40, -50, -62, -75, -100, -126, -133, -40.25, 60]


@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-6, 2.0 ** 100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,rot,inter", [(128, 128, False), (128, 128, True), (96, 32, False), (256, 256, False),
                                           (64, 0, False), (64, 6, False), (16, 16, False)])
def test_norms_near_the_ends_of_the_type(sv, h, dtype, dim, rot, inter, eps):  # noqa: F811
    """Heads of one size beside heads of another in every warp, for q and k: within the bound of ordinary
    heads, as a power of two costs no rounding (values below 2^-126 enter without loss)."""
    import torch

    rng = np.random.default_rng(dim + rot)
    heads, dt = len(ENDS), _dtype(dtype)
    size = np.array([2.0 ** e for e in ENDS])[:, None] * rng.choice([1.0, -1.0, 0.75, 0.5], size=(heads, dim))
    lone = size.copy()
    lone[:, 1:] = 0.0  # one value a head, at an end of it
    both = np.stack([size, lone], 0)[None].astype(np.float32)  # [1, 2 rows, heads, dim]
    x_t = torch.from_numpy(both).to(dt).cuda()
    x = _np(x_t)
    w = [torch.from_numpy(rng.normal(size=dim).astype(np.float32)).to(dt).cuda() for _ in range(2)]
    inv = (10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32) if rot else None
    kc = torch.zeros((1, heads, 2, dim), dtype=dt, device="cuda")
    vc = kc.clone()
    ref_k, ref_v = _np(kc), _np(vc)
    tables, lens = np.zeros((1, 1), np.int32), np.array([2], np.int32)
    with np.errstate(invalid="ignore"):
        q_out, _, _, (q_mag, k_mag) = S.append_norm(ref_k, ref_v, tables, lens, x, x, q=x, q_norm=_np(w[0]), k_norm=_np(w[1]),
                                                    eps=float(np.float32(eps)), inv_freq=inv, interleaved=inter)
    got = sv.specv_cache_append_norm(h, kc, vc, _dev(tables), _dev(lens), x_t, x_t, q=x_t, q_norm=w[0], k_norm=w[1], eps=eps,
                                     inv_freq=None if inv is None else _dev(inv), interleaved=inter)
    qq = x_t.clone()  # in place: what a head needs is still there when its turn comes
    sv.specv_cache_append_norm(h, kc, vc, _dev(tables), _dev(lens), x_t, x_t, q=qq, q_norm=w[0], k_norm=w[1], eps=eps,
                               inv_freq=None if inv is None else _dev(inv), interleaved=inter, out={"q_out": qq})
    torch.cuda.synchronize()
    np.testing.assert_array_equal(_np(qq), _np(got["q_out"]))
    half, least = (BF16_HALF, 2.0 ** -134) if dtype == "bf16" else (F32_HALF, 2.0 ** -150)
    # a result below the normal numbers rounds by half of the smallest number there is (`least`); so may each of up to four
    # fp32 products and two sums that make it (2^-150 each), of which those before the head's factor are as much larger
    # as that is: at most 1 / sqrt(eps), and heads whose mean is below 2^-90 are scaled before
    least = least + 8 * 2.0 ** -150 * max(1.0, eps ** -0.5 if eps >= 2.0 ** -90 else 0.0)
    for g, ref, mag in ((got["q_out"], q_out, q_mag), (kc, ref_k, k_mag)):
        # (2^-134, half of 2^-133, is no value of bf16 but becomes zero: with eps 0 such a head is 0 / 0, for both)
        np.testing.assert_array_equal(np.isnan(_np(g)), np.isnan(ref))
        bad = ~np.isnan(ref) & ~(np.abs(_np(g) - ref) <= S.append_norm_bound(ref, mag, dim, half) + least)
        assert not bad.any(), (np.argwhere(bad)[:4], _np(g)[bad][:4], ref[bad][:4])


@pytest.mark.parametrize("dim", [64, 48])
@pytest.mark.parametrize("rot", [0, 6])
def test_a_head_that_is_no_number_takes_no_other(sv, h, dim, rot):  # noqa: F811
    """Zeros with eps 0, an infinity and a NaN: their own heads, as the formula has them."""
    import torch

    x = torch.ones((1, 1, 6, dim), device="cuda")
    x[0, 0, 1] = 0.0
    x[0, 0, 2, 7], x[0, 0, 3, 9] = float("inf"), float("nan")
    x[0, 0, 4] *= 2.0 ** 127
    x[0, 0, 5] *= 2.0 ** -126
    kc = torch.zeros((1, 6, 1, dim), device="cuda")
    vc, one = kc.clone(), torch.ones(1, dtype=torch.int32, device="cuda")
    inv = torch.zeros(rot // 2, device="cuda") if rot else None
    sv.specv_cache_append_norm(h, kc, vc, one[:, None] - 1, one, x, x, k_norm=torch.full((dim,), 2.0, device="cuda"), eps=0.0,
                               inv_freq=inv)
    k = _np(kc)[0, :, 0]
    for i in (0, 4, 5):
        assert np.abs(k[i] - 2).max() <= 2 * 2.0 ** -20, i
    assert np.isnan(k[1]).all() and np.isnan(k[3]).all()
    assert np.isnan(k[2, 7]) and (k[2, 8:] == 0).all()
