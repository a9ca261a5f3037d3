"""Pins of the language-model oracle (oracle.lm): hand values, invariants and finite differences."""
import math

import numpy as np
import pytest

from oracle import e4m3 as E
from oracle import lm


def test_rmsnorm_by_hand():
    y, r = lm.rmsnorm(np.array([[3.0, 4.0, 0.0, 0.0]]), np.array([1.0, 2.0, 1.0, 1.0]), 0.0)
    assert r[0] == pytest.approx(0.4)  # sqrt(25 / 4) = 2.5
    assert np.allclose(y, [[1.2, 3.2, 0.0, 0.0]])


def test_rmsnorm_gradients_by_differences():
    rng = np.random.default_rng(0)
    h, g, w = rng.standard_normal((3, 8)), rng.standard_normal(8), rng.standard_normal((3, 8))
    dh, dg = lm.rmsnorm_bwd(w, h, g, 1e-3)
    loss = lambda h, g: float((lm.rmsnorm(h, g, 1e-3)[0] * w).sum())  # noqa: E731
    e = 1e-6
    for i, j in ((0, 0), (1, 5), (2, 7)):
        d = np.zeros_like(h)
        d[i, j] = e
        assert (loss(h + d, g) - loss(h - d, g)) / (2 * e) == pytest.approx(dh[i, j], rel=1e-6, abs=1e-9)
    for j in range(8):
        d = np.zeros(8)
        d[j] = e
        assert (loss(h, g + d) - loss(h, g - d)) / (2 * e) == pytest.approx(dg[j], rel=1e-6, abs=1e-9)
    assert np.allclose(lm.rmsnorm_bwd(w, h, g, 1e-3, dh_in=h)[0], dh + h)


def test_block_scale_values():
    assert lm.block_scale(0.0) == 1.0
    assert lm.block_scale(448.0) == 1.0 or abs(lm.block_scale(448.0) - 1) <= 2.0 ** -23
    assert lm.block_scale(2.0) == 224.0
    assert lm.block_scale(1e-38) == 2.0 ** 100 and lm.block_scale(np.float32(1e-45)) == 2.0 ** 100


def test_casts_land_on_the_top_code_and_keep_tiles_apart():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 300)).astype(np.float32)
    x[2, 130] = 1000.0
    x[3, :128] = 0.0
    q, s = lm.cast_rows(x)
    assert s.shape == (3, 5) and s[0, 3] == 1.0 and not q[3, :128].any()
    v = lm.decode(q)
    for r in range(5):
        for j in range(3):
            if r != 3 or j:
                assert np.abs(v[r, 128 * j:128 * (j + 1)]).max() == 448.0
    half_step = np.maximum(np.abs(x * np.repeat(s.T, 128, 1)[:, :300]) * 2.0 ** -4, 2.0 ** -10)
    assert (np.abs(v - x * np.repeat(s.T, 128, 1)[:, :300]) <= half_step * (1 + 1e-5)).all()
    x[0, 5] = np.nan
    q2, s2 = lm.cast_rows(x)
    assert q2[0, 5] & 0x7F == 0x7F and (np.delete(q2[0], 5) & 0x7F != 0x7F).all() and np.isfinite(s2).all()


def test_square_cast_is_one_scale_per_tile():
    rng = np.random.default_rng(2)
    w = rng.standard_normal((200, 140)).astype(np.float32)
    q, s = lm.cast_square(w)
    assert s.shape == (2, 2)
    for i in range(2):
        for j in range(2):
            t = w[128 * i:128 * (i + 1), 128 * j:128 * (j + 1)]
            assert s[i, j] == lm.block_scale(np.abs(t).max())
    assert np.array_equal(q[130, 129], E.e4m3_encode(np.float64(np.float32(w[130, 129] * s[1, 1]))))


def test_linear_on_values_that_codes_hold_exactly():
    rng = np.random.default_rng(3)
    x = rng.integers(-7, 8, (4, 256)).astype(np.float32)
    w = rng.integers(-7, 8, (136, 256)).astype(np.float32)
    x[:, ::128], w[::128, ::128] = 7, 7  # every tile's amax is 7: 448 / 7 = 64, a power of two
    w[0:128, 0], w[128:, 128] = 7, 7
    xq, sx = lm.cast_rows(x)
    wq, sw = lm.cast_square(w)
    assert np.allclose(lm.block_linear(xq, sx, wq, sw, np.ones(136)), x.astype(np.float64) @ w.T + 1, rtol=1e-6)


def test_linear_gradients_match_the_exact_ones_to_the_casts():
    rng = np.random.default_rng(4)
    M, N, K = 150, 136, 272
    x, w, dy = (rng.standard_normal(s).astype(np.float32) for s in ((M, K), (N, K), (M, N)))
    wq, sw = lm.cast_square(w)
    xt, sxt = lm.cast_rows(x.T)
    dx, dw, db = lm.block_linear_bwd(dy, wq, sw, xt, sxt)
    for got, ref in ((dx, dy.astype(np.float64) @ w), (dw, dy.T.astype(np.float64) @ x)):
        # each factor is off by at most 2^-4 of itself, on average far less
        assert np.linalg.norm(got - ref) / np.linalg.norm(ref) < 0.06
    assert np.allclose(db, dy.astype(np.float64).sum(0))


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_properties(interleaved):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, 3, 2, 24))
    f = lm.rope_frequencies(16)
    pos = np.array([[0, 5, 9], [1, 100000, -4]])
    c, s = lm.rope_cos_sin(pos, f)
    y = lm.rope(x, c, s, 16, interleaved, mscale=1.5)
    assert np.allclose(y[0, 0, :, :16], 1.5 * x[0, 0, :, :16]) and np.array_equal(y[..., 16:], x[..., 16:])
    assert np.allclose(np.linalg.norm(y[..., :16], axis=-1), 1.5 * np.linalg.norm(x[..., :16], axis=-1))
    # the gradient is the adjoint: <R x, g> = <x, R^T g> on the rotated part
    g = rng.standard_normal(x.shape)
    b = lm.rope(g, c, s, 16, interleaved, mscale=1.5, transposed=True)
    assert np.sum(y * g) == pytest.approx(np.sum(x * b), rel=1e-12)
    # scores depend on position differences alone
    q = lm.rope(x, *lm.rope_cos_sin(pos, f), 16, interleaved)
    q7 = lm.rope(x, *lm.rope_cos_sin(pos + 7, f), 16, interleaved)
    assert np.allclose(np.einsum("bshd,bthd->bhst", q, q), np.einsum("bshd,bthd->bhst", q7, q7))


def test_rope_scalings():
    f = lm.rope_frequencies(8)
    assert np.allclose(f, [1.0, 0.1, 0.01, 0.001])
    assert np.allclose(lm.rope_frequencies(8, scaling="linear", factor=4.0), f / 4)
    g = lm.rope_frequencies(8, scaling="by_parts", factor=4.0, orig_len=2 * math.pi * 50, low=1.0, high=4.0)
    # 50, 5, 0.5 and 0.05 turns within the trained length: kept, kept, interpolated, interpolated
    assert np.allclose(g, [1.0, 0.1, 0.0025, 0.00025])
    h = lm.rope_frequencies(8, scaling="by_parts", factor=4.0, orig_len=2 * math.pi * 25, low=1.0, high=4.0)
    assert h[1] == pytest.approx(0.1 * (0.5 + 0.5 / 4))  # 2.5 turns: halfway


def test_rope_exact_frequencies_and_angles():
    """The 80-digit frequencies against the double ones, 2 pi against known digits, and the angle of a far position
    against whole-number arithmetic: theta = 2^24 and rot = 4 make f_1 = 2^-12 exactly."""
    assert str(lm._two_pi(60))[:42] == "6.2831853071795864769252867665590057683943"
    for kw in (dict(), dict(scaling="linear", factor=8.0), dict(scaling="by_parts", factor=8.0, orig_len=4096.0, high=32.0)):
        exact, double = lm.rope_turns_exact(32, **kw), lm.rope_frequencies(32, **kw)
        assert np.allclose([float(e) for e in exact], double / (2 * np.pi), rtol=1e-14, atol=0)
    turns = lm.rope_turns_exact(4, theta=2.0 ** 24)
    p = np.array([3, (1 << 40) + 7, -5])
    cos, sin = lm.rope_cos_sin_exact(p, turns)
    assert np.allclose(cos[[0, 2], 0], np.cos([3.0, -5.0]), atol=1e-15) and np.allclose(sin[[0, 2], 0], np.sin([3.0, -5.0]), atol=1e-15)
    # p 2^-12 at p = 2^40 + 7 is 2^28 + 7 2^-12: exact in a double, whose cosine math.cos reduces exactly
    assert abs(cos[1, 1] - math.cos(2.0 ** 28 + 7 * 2.0 ** -12)) < 1e-14 and abs(sin[1, 1] - math.sin(2.0 ** 28 + 7 * 2.0 ** -12)) < 1e-14
