"""Pins of oracle/int8.py against values derived by hand and against other evaluations of the definitions."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import int8 as o8


def test_quantizer_hand_derived():
    # a = 127: r = 1, s = 1; ties go to the even code; the maximum is +-127
    q, s = o8.quantize(np.array([[127.0, -127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 0.49999997]]))
    assert q.tolist() == [[127, -127, 0, 2, 2, 0, -2, 126, 0]] and s.tolist() == [1.0]
    # a = 63.5: r = 2 exactly, s = 0.5
    q, s = o8.quantize(np.array([[63.5, 0.25, 0.75, -31.75]]))
    assert q.tolist() == [[127, 0, 2, -64]] and s.tolist() == [0.5]
    # the floor: a row below 2^-96 is divided by 2^-96
    q, s = o8.quantize(np.array([[2.0 ** -97, 0.0]]))
    assert q.tolist() == [[64, 0]] and s[0] == np.float32(2.0 ** -96 / 127)
    # smoothing rounds once to fp32 before the maximum
    q, s = o8.quantize(np.array([[2.0, 10.0]]), np.array([3.0, 0.1], np.float32))
    assert q.tolist() == [[127, 21]] and s[0] == np.float32(6.0 / 127)
    q, s = o8.quantize(np.array([[1.0, np.nan], [np.inf, 2.0], [3.0, 4.0]]))
    assert np.isnan(s[:2]).all() and (q[:2] == 0).all() and np.isfinite(s[2])


def test_quantizer_roundings_are_single():
    """s and r are the fp32 values nearest to the exact quotients, by exact fractions."""
    rng = np.random.default_rng(0)
    for a in (rng.random(300) * 10.0 ** rng.integers(-20, 20, 300)).astype(np.float32):
        _, s = o8.quantize(np.array([[float(a), 0.0]]))
        for got, want in ((s[0], Fraction(float(a)) / 127), (o8._f32(127.0 / float(a)), 127 / Fraction(float(a)))):
            g = np.float32(got)
            err = abs(Fraction(float(g)) - want)
            for other in (np.nextafter(g, np.float32(np.inf)), np.nextafter(g, np.float32(0))):
                assert err <= abs(Fraction(float(other)) - want)


def test_codes_are_nearest_values():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 200))
    q, s = o8.quantize(x.astype(np.float32).astype(np.float64))
    # the factor and the product are rounded: at most 2 ulp of a value up to 127 beside half a step
    assert (np.abs(q * s[:, None] - x) <= s[:, None] * (0.5 + 127 * 2.0 ** -22) + 1e-7).all()
    assert (np.abs(q).max(axis=1) == 127).all()


def test_product_by_loops():
    rng = np.random.default_rng(2)
    qX, qW = rng.integers(-127, 128, (3, 5)), rng.integers(-127, 128, (4, 5))
    sX, sW, b = rng.random(3), rng.random(4), rng.standard_normal(4)
    y = o8.product(qX, sX, qW, sW, b)
    for m in range(3):
        for n in range(4):
            assert y[m, n] == pytest.approx(sum(int(qX[m, k]) * int(qW[n, k]) for k in range(5)) * sX[m] * sW[n] + b[n], rel=1e-14)


def test_pack_reproduces_planted_codes():
    """Columns that are exact multiples of their scale give back codes and scales, in [N][K] order."""
    rng = np.random.default_rng(3)
    codes = rng.integers(-127, 128, (6, 40))
    codes[:, 0] = 127
    sc = 2.0 ** rng.integers(-8, 8, 6)
    _, inv, q, s = o8.pack_weights((codes * sc[:, None]).T)
    np.testing.assert_array_equal(q[:, :40], codes)
    np.testing.assert_array_equal(s, sc)
    assert q.shape == (6, 128) and (q[:, 40:] == 0).all() and (inv == 1).all()


def test_group_norm_by_loops():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, 3, 6)) + 5
    gamma, beta = rng.standard_normal(6), rng.standard_normal(6)
    y, mean, var = o8.group_norm(x, 3, gamma, beta, 0.1, "none")
    for b in range(2):
        for g in range(3):
            v = [x[b, i, c] for i in range(3) for c in (2 * g, 2 * g + 1)]
            m = sum(v) / 6
            w = sum((t - m) ** 2 for t in v) / 6
            for i in range(3):
                for c in (2 * g, 2 * g + 1):
                    assert y[b, i, c] == pytest.approx((x[b, i, c] - m) / (w + 0.1) ** 0.5 * gamma[c] + beta[c], rel=1e-12)
                    assert mean[b, 0, c] == pytest.approx(m) and var[b, 0, c] == pytest.approx(w)


def test_group_norm_against_torch():
    import torch

    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, 10, 12))
    t = torch.nn.functional.group_norm(torch.from_numpy(x).permute(0, 2, 1), 4, eps=1e-3).permute(0, 2, 1).numpy()
    np.testing.assert_allclose(o8.group_norm(x, 4, eps=1e-3)[0], t, rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(o8.silu(x), torch.nn.functional.silu(torch.from_numpy(x)).numpy(), rtol=1e-12)
    np.testing.assert_allclose(o8.gelu(x), torch.nn.functional.gelu(torch.from_numpy(x)).numpy(), rtol=1e-10, atol=1e-13)
    assert o8.silu(np.array([-1e4]))[0] == 0.0
