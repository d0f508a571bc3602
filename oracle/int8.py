"""The 8-bit layer (W8A8) and the channels-last group norm, in fp64 and exact integers, from their formulas.

    quantize  v = fp32(x inv_s); a = max(max |v|, 2^-96); s = fp32(a / 127); r = fp32(127 / a);
              q = round_half_even(fp32(v r)); a row with a NaN or an infinity: s = NaN, q = 0
    product   Y = (sum_k qX qW) s_X s_W + bias, the sum in integers, the rest in fp64
    norm      y = act((x - mean) / sqrt(var + eps) gamma + beta) over a group's positions and channels

The smoothed 8-bit layer with per-token and per-channel scales is the ch3chohch3.github.io post "从 Smooth Quant
到 SVD Quant", section "Smooth Quant（W8A8）".
"""
from __future__ import annotations

import numpy as np
from scipy.special import erfc

FLOOR = 2.0 ** -96


def ld(K: int) -> int:
    return -(-K // 128) * 128


def _f32(x):
    """One rounding of fp64 values to fp32.  Exact products of two fp32 values fit fp64, and an fp64 quotient of two
    fp32 values rounds to the same fp32 as the exact quotient (53 >= 2 * 24 + 2 bits)."""
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def quantize(x, inv_s=None):
    """(codes int8 [M][K], scales fp32 [M]) of fp32 / bf16 values given as fp64 [M][K]."""
    with np.errstate(over="ignore", invalid="ignore"):
        v = np.asarray(x, np.float64)
        if inv_s is not None:
            v = _f32(v * np.asarray(inv_s, np.float64))
        bad = ~np.isfinite(v).all(axis=1)
        a = np.maximum(np.abs(np.where(np.isfinite(v), v, 0.0)).max(axis=1), FLOOR)
        r = _f32(127.0 / a)
        q = np.rint(_f32(np.where(bad[:, None], 0.0, v) * r[:, None]))
    s = _f32(a / 127.0)
    s[bad] = np.nan
    return q.astype(np.int8), s.astype(np.float32)


def pack_weights(W, act_absmax=None, alpha=0.5):
    """(s, inv_s fp32 [K], codes int8 [N][ld(K)], scales fp32 [N]) of W [K][N] (fp64 values of bf16 weights)."""
    W = np.asarray(W, np.float64)
    K, N = W.shape
    s = np.ones(K, np.float32)
    if act_absmax is not None:
        a, w = np.maximum(np.asarray(act_absmax, np.float64), 1e-5), np.maximum(np.abs(W).max(axis=1), 1e-5)
        s = (a ** alpha / w ** (1.0 - alpha)).astype(np.float32)
    What = s.astype(np.float64)[:, None] * W
    sW = (np.abs(What).max(axis=0) / 127.0).astype(np.float32)
    d = np.where(sW == 0, 1.0, sW.astype(np.float64))
    q = np.clip(np.rint(What / d), -127, 127) * (sW != 0)
    out = np.zeros((N, ld(K)), np.int8)
    out[:, :K] = q.T.astype(np.int8)
    return s, (np.float32(1.0) / s).astype(np.float32), out, sW


def gelu(y):
    return y * erfc(-y / np.sqrt(2.0)) / 2.0


def silu(y):
    with np.errstate(over="ignore"):
        return y / (1.0 + np.exp(-y))


def product(qX, sX, qW, sW, bias=None):
    """fp64 [M][N]; the integer sums are exact in fp64 products (|sum| < 2^31)."""
    acc = np.asarray(qX, np.float64) @ np.asarray(qW, np.float64).T
    y = acc * np.asarray(sX, np.float64)[:, None] * np.asarray(sW, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64)


def group_norm(x, groups, gamma=None, beta=None, eps=1e-5, act="none"):
    """fp64 [B][S][C] of x [B][S][C]; also (mean, var) as [B][1][C]."""
    x = np.asarray(x, np.float64)
    B, S, C = x.shape
    g = x.reshape(B, S, groups, C // groups)
    mean = g.mean(axis=(1, 3), keepdims=True)
    var = ((g - mean) ** 2).mean(axis=(1, 3), keepdims=True)
    y = ((g - mean) / np.sqrt(var + eps)).reshape(B, S, C)
    y = y * (1.0 if gamma is None else np.asarray(gamma, np.float64)) + (0.0 if beta is None else np.asarray(beta, np.float64))
    wide = lambda t: np.broadcast_to(t, (B, 1, groups, C // groups)).reshape(B, 1, C)  # noqa: E731
    return {"none": lambda t: t, "silu": silu, "gelu": gelu}[act](y), wide(mean), wide(var)
