"""Pins of oracle/fp8.py: values worked out from the definitions, and the gradient against differences (CPU)."""
import numpy as np
import pytest

from oracle import fp8 as o


def test_e4m3_values():
    """Named points of the format, and the order of its codes."""
    assert o.decode([0x00, 0x01, 0x07, 0x08, 0x38, 0x40, 0x7E]).tolist() == [0, 2 ** -9, 7 * 2 ** -9, 2 ** -6, 1, 2, 448]
    assert o.decode([0xB8])[0] == -1.0 and np.isnan(o.decode([0x7F])[0])
    assert (np.diff(o.VALUES) > 0).all()


def test_encode_rounds_to_nearest_even():
    assert np.array_equal(o.encode(o.VALUES), np.arange(127))
    mids = (o.VALUES[1:] + o.VALUES[:-1]) / 2
    assert (o.encode(mids) % 2 == 0).all()
    assert np.array_equal(o.encode(np.nextafter(mids, 0)), np.arange(126))
    assert np.array_equal(o.encode(np.nextafter(mids, 1e9)), np.arange(1, 127))
    assert o.encode(460.0) == 126 and o.encode(-1.0) == 0xB8 and o.encode(-0.0) == 0x80


def test_quantize_by_hand():
    x = np.zeros((2, 130))
    x[0, :3] = [448.0, 1.0, -17.0]  # r = 1: 17 lies between 16 and 18, a tie: the even code (16)
    x[0, 129] = 0.875  # alone in its block: the largest magnitude is 448 s
    x[1, 5] = np.nan
    q, s = o.quantize(x)
    assert s[0, 0] == 1.0 and o.decode(q[0, :3]).tolist() == [448, 1, -16]
    assert s[1, 0] == np.float32(0.875 / 448) and q[0, 129] == 126
    assert np.isnan(s[0, 1]) and (q[1] == 0).all() and s[1, 1] == np.float32(2.0 ** -96 / 448)
    assert q.shape == (2, 256) and (q[:, 130:] == 0).all()


def test_pack_and_product_small():
    rng = np.random.default_rng(0)
    W = rng.standard_normal((200, 150))
    q, s = o.pack_weights(W)
    assert q.shape == (150, 256) and s.shape == (2, 2)
    w = o.values(q, s, 128)[:, :200].T
    assert np.abs(w - W).max() <= np.abs(W).max() * 2.0 ** -4  # half a step of the largest binade
    x = rng.standard_normal((3, 200))
    qx, sx = o.quantize(x)
    y = o.product(qx, sx, q, s)
    ref = np.zeros((3, 150))
    for m in range(3):
        for n in range(150):
            for b in range(2):
                k = slice(128 * b, 128 * b + 128)
                ref[m, n] += float(sx[b, m]) * float(s[n // 128, b]) * (o.decode(qx[m, k]) * o.decode(q[n, k])).sum()
    assert np.allclose(y, ref, rtol=1e-13, atol=1e-13)
    assert np.abs(y - x @ W).max() < 0.1 * np.abs(x @ W).max()


def test_layer_norm_by_hand():
    y, mean, rstd = o.layer_norm(np.array([[1.0, 3.0]]), np.array([0.5, 0.0]), np.array([1.0, 2.0]), eps=0.0, one_plus=True)
    assert mean[0] == 2.0 and rstd[0] == 1.0 and y.tolist() == [[-0.5, 3.0]]


@pytest.mark.parametrize("C", [1, 2, 7, 40])
@pytest.mark.parametrize("one_plus", [False, True])
def test_gradient_against_differences(C, one_plus):
    rng = np.random.default_rng(C)
    x, v = rng.standard_normal((5, C)) * 2 + 1, rng.standard_normal((5, C))
    gamma, beta, eps = rng.standard_normal(C), rng.standard_normal(C), 1e-2

    def f(x, gamma, beta):
        return (o.layer_norm(x, gamma, beta, eps, one_plus)[0] * v).sum()

    _, mean, rstd = o.layer_norm(x, gamma, beta, eps, one_plus)
    dx, dgz, dy = o.layer_norm_grad(v, x, mean, rstd, gamma, one_plus)
    h = 1e-6
    for grad, i in ((dx, 0), (dgz.sum(0), 1), (dy.sum(0), 2)):
        for at in np.ndindex(grad.shape):
            args = [x, gamma, beta]
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[i][at] += h
            lo[i][at] -= h
            assert abs((f(*hi) - f(*lo)) / (2 * h) - grad[at]) < 1e-6 * (1 + abs(grad[at]))
