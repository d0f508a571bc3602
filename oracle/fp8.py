"""The block-scaled E4M3 layer and the layer norm with its gradient, in fp64, from their formulas.

    quantize  per row and block of 128: a = max(max |x|, 2^-96); s = fp32(a / 448); r = fp32(448 / a);
              q = E4M3(fp32(x r)); a block with a NaN or an infinity: s = NaN, q = 0
    product   Y = sum over blocks s_X s_W (sum qX qW) + bias
    norm      z = (x - mean) / sqrt(var + eps); y = z w + beta, w = gamma or 1 + gamma
    gradient  g = dy w; dx = rstd (g - mean(g) - z mean(g z)); dgamma = sum dy z; dbeta = sum dy

E4M3 is the finite 8-bit format with 4 exponent bits (bias 7) and 3 of mantissa: code c < 127 stands for
(c % 8) 2^-9 where c < 8 and (8 + c % 8) 2^(c / 8 - 10) above; bit 7 is the sign, 127 a NaN.
"""
from __future__ import annotations

import numpy as np

FLOOR = 2.0 ** -96
VALUES = np.array([c * 2.0 ** -9 if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - 10) for c in range(127)])
_MIDS = (VALUES[1:] + VALUES[:-1]) / 2


def blocks(n: int) -> int:
    return -(-n // 128)


def ld(K: int) -> int:
    return blocks(K) * 128


def _f32(x):
    """One rounding of fp64 values to fp32 (exact products of two fp32 values fit fp64, and an fp64 quotient of two fp32
    values rounds to the same fp32 as the exact one)."""
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def encode(v):
    """E4M3 codes (uint8) of fp64 values: the nearest magnitude, ties to the even code, saturating at 448."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    i = np.searchsorted(_MIDS, a, side="left")
    j = np.minimum(i, len(_MIDS) - 1)
    i = i + ((a == _MIDS[j]) & (i % 2 == 1))
    return (i + 128 * np.signbit(v)).astype(np.uint8)


def decode(codes):
    c = np.asarray(codes, np.uint8).astype(np.int64)
    out = np.append(VALUES, np.nan)[c & 127]
    return np.where(c >= 128, -out, out)


def quantize(x):
    """(codes uint8 [M][ld(K)], scales fp32 [blocks(K)][M]) of fp32 / bf16 values given as fp64 [M][K]."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    t = np.zeros((M, ld(K)))
    t[:, :K] = x
    t = t.reshape(M, -1, 128)
    bad = ~np.isfinite(t).all(axis=2)
    t = np.where(bad[:, :, None], 0.0, t)
    a = np.maximum(np.abs(t).max(axis=2), FLOOR)
    q = encode(_f32(t * _f32(448.0 / a)[:, :, None])).reshape(M, -1)
    q = np.where(np.repeat(bad, 128, axis=1), 0, q).astype(np.uint8)
    q[:, K:] = 0
    s = _f32(a / 448.0)
    s[bad] = np.nan
    return q, np.ascontiguousarray(s.T.astype(np.float32))


def pack_weights(W):
    """(codes uint8 [N][ld(K)], scales fp32 [blocks(N)][blocks(K)]) of W [K][N] (fp64 values of bf16 weights)."""
    K, N = W.shape
    t = np.zeros((ld(N), ld(K)))
    t[:N, :K] = np.asarray(W, np.float64).T
    t = t.reshape(blocks(N), 128, blocks(K), 128)
    s = (np.abs(t).max(axis=(1, 3)) / 448.0).astype(np.float32)
    d = np.where(s == 0, 1.0, s.astype(np.float64))[:, None, :, None]
    q = np.where((s == 0)[:, None, :, None], 0, encode(t / d))
    return np.ascontiguousarray(q.reshape(ld(N), ld(K))[:N]).astype(np.uint8), s


def values(q, s, rows_per_scale):
    """fp64 values of codes [n][ld] under scales [n / rows_per_scale][blocks]."""
    w = np.repeat(np.repeat(np.asarray(s, np.float64), rows_per_scale, axis=0)[:q.shape[0]], 128, axis=1)
    with np.errstate(invalid="ignore"):
        return decode(q) * w


def product(qX, sX, qW, sW, bias=None, magnitude=False):
    """fp64 [M][N] of codes qX [M][ld], sX [blocks][>= M], qW [N][ld], sW; `magnitude`: of the absolute values."""
    M = qX.shape[0]
    x, w = values(qX, np.asarray(sX)[:, :M].T, 1), values(qW, sW, 128)
    if magnitude:
        return np.abs(x) @ np.abs(w).T + (0.0 if bias is None else np.abs(np.asarray(bias, np.float64)))
    return x @ w.T + (0.0 if bias is None else np.asarray(bias, np.float64))


def _weight(gamma, one_plus):
    return 1.0 if gamma is None else np.asarray(gamma, np.float64) + (1.0 if one_plus else 0.0)


def layer_norm(x, gamma=None, beta=None, eps=1e-5, one_plus=False):
    """(y, mean, rstd) in fp64 of x [..., C]; gamma and beta broadcast against x."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(axis=-1, keepdims=True) + eps)
    y = (x - mean) * rstd * _weight(gamma, one_plus) + (0.0 if beta is None else np.asarray(beta, np.float64))
    return y, mean[..., 0], rstd[..., 0]


def layer_norm_grad(dy, x, mean, rstd, gamma=None, one_plus=False):
    """(dx, dy z, dy) in fp64; dgamma and dbeta are the last two summed over the rows that share gamma and beta."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    r = np.asarray(rstd, np.float64)[..., None]
    z = (x - np.asarray(mean, np.float64)[..., None]) * r
    g = dy * _weight(gamma, one_plus)
    dx = r * (g - g.mean(axis=-1, keepdims=True) - z * (g * z).mean(axis=-1, keepdims=True))
    return dx, dy * z, dy
