"""GPU tests of the 8-bit layer (W8A8) against oracle/int8.py (fp64, exact integers).

Bounds, derived from the formulas (u = 2^-24, one fp32 rounding):
* codes and scales: equal, bit for bit (every deciding operation is one defined rounding);
* products in fp32: conversion of the integer sum, two scale products, the bias addition: at most 4 roundings, each of
  a value no larger than |p| + |b| with p the product term: 5 u (|p| + |b|);
* GELU: slope at most 1.13, its own relative error 2e-5 (the fit's documented bound);
* bf16: half a step, 2^-8 / 2 of the value (and of the smallest normal below it).
"""
import numpy as np
import pytest

from gpu_helpers import log

from bit_diffusion_model_amd import svdq
from oracle import int8 as o8

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _torch():
    import torch

    return torch


def make_x(M, K, dtype, seed, pad=0):
    """Rows of normals with outlier channels, each row of its own magnitude, as a (possibly padded) device tensor."""
    torch = _torch()
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K)) * 10.0 ** rng.uniform(-3, 3, (M, 1))
    x[:, rng.choice(K, max(1, K // 50), replace=False)] *= 30.0
    t = torch.from_numpy(x.astype(np.float32)).to("cuda:0").to(dtype)
    buf = torch.full((M, K + pad), 1e30, dtype=dtype, device="cuda:0")
    buf[:, :K] = t
    return buf[:, :K]


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def tol_product(p, bias, ydtype):
    lin = 5 * U * (np.abs(p) + (0.0 if bias is None else np.abs(bias)))
    y = p if bias is None else p + bias
    if ydtype == svdq.F32:
        return lin + 1e-37
    if ydtype == svdq.BF16:
        return lin + 2.0 ** -8 * np.abs(y) + 1e-37
    return 1.13 * lin + (2e-5 + 2.0 ** -8) * np.abs(o8.gelu(y)) + 1e-37


def check_product(Y, qX, sX, qW, sW, bias, ydtype, what):
    p = o8.product(qX, sX, qW, sW)
    ref = p if bias is None else p + bias
    ref = o8.gelu(ref) if ydtype == svdq.BF16_GELU else ref
    got = host(Y)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), what
    err = np.abs(got - ref)[~nan]
    tol = np.broadcast_to(tol_product(p, bias, ydtype), ref.shape)[~nan]
    assert (err <= tol).all(), f"{what}: worst {np.max(err / tol)} of the bound"


# one token to many, one value to rows longer than what a block holds; strides that allow and forbid wide loads
@pytest.mark.parametrize("M,K,pad", [(1, 1, 0), (1, 7, 0), (3, 8, 0), (5, 127, 1), (4, 128, 0), (2, 129, 7), (9, 512, 8),
                                     (7, 1000, 0), (5, 1025, 0), (6, 3072, 16), (3, 4097, 0), (2, 8200, 8),
                                     (2, 16384, 0), (2, 20001, 3)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("smooth", [False, True])
def test_quantizer_bit_exact(M, K, pad, dt, smooth):
    torch = _torch()
    X = make_x(M, K, {"bf16": torch.bfloat16, "f32": torch.float32}[dt], M * 1000 + K, pad)
    inv = (0.2 + np.random.default_rng(K).random(K)).astype(np.float32) if smooth else None
    qX, sX = svdq.quantize_act_int8(X, None if inv is None else torch.from_numpy(inv).to("cuda:0"))
    q, s = o8.quantize(host(X), inv)
    assert np.array_equal(qX.cpu().numpy()[:, :K], q) and (qX.cpu().numpy()[:, K:] == 0).all()
    assert np.array_equal(sX.cpu().numpy(), s)


def test_quantizer_special_rows():
    """Rows of zeros, of the smallest and largest values, exact ties, NaN and infinities (whose rows alone are lost)."""
    torch = _torch()
    K = 300
    x = np.zeros((9, K), np.float32)
    x[1, 5] = 1e-45
    x[2, :] = np.linspace(-1e-38, 1e-38, K)
    x[3, :] = np.float32(3.4e38)
    x[4, :255] = np.arange(-127, 128) / 2.0  # 127/a = 2: the halves are ties
    x[4, 254] = 63.5
    x[5, 17] = np.nan
    x[6, 250] = -np.inf
    x[7, :] = -5.0
    x[8, 0] = 2.0 ** -97
    X = torch.from_numpy(x).to("cuda:0")
    qX, sX = svdq.quantize_act_int8(X)
    q, s = o8.quantize(x.astype(np.float64))
    assert np.array_equal(qX.cpu().numpy()[:, :K], q)
    np.testing.assert_array_equal(sX.cpu().numpy(), s)
    assert np.isnan(s[5]) and np.isnan(s[6]) and (q[0] == 0).all()
    lin = svdq.Int8Linear(np.ones((40, svdq.int8_ld(K)), np.int8) * (np.arange(svdq.int8_ld(K)) < K).astype(np.int8),
                          np.ones(40, np.float32), K)
    Y = lin.forward(X).cpu().numpy()
    assert np.isnan(Y[5]).all() and np.isnan(Y[6]).all() and np.isfinite(Y[[0, 1, 2, 4, 7, 8]]).all()


def weights(N, K, seed, bias):
    rng = np.random.default_rng(seed)
    qW = np.zeros((N, svdq.int8_ld(K)), np.int8)
    qW[:, :K] = rng.integers(-127, 128, (N, K))
    sW = (10.0 ** rng.uniform(-4, 0, N)).astype(np.float32)
    return qW, sW, (rng.standard_normal(N) * 3).astype(np.float32) if bias else None


SHAPES = [(1, 1, 1), (1, 64, 33), (2, 128, 1000), (3, 3072, 40), (4, 130, 4097), (16, 640, 257), (17, 320, 64),
          (33, 1000, 100), (63, 256, 31), (64, 384, 512), (65, 1153, 129), (128, 12288, 64), (200, 77, 200),
          (255, 512, 513), (257, 640, 1280), (300, 3072, 300), (1030, 256, 770), (700, 100, 2100), (1, 131072, 3)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("yd,bias", [("f32", True), ("bf16", False), ("gelu", True)])
def test_product(M, K, N, yd, bias):
    torch = _torch()
    ydtype = {"f32": svdq.F32, "bf16": svdq.BF16, "gelu": svdq.BF16_GELU}[yd]
    rng = np.random.default_rng(M + K + N)
    qX = rng.integers(-127, 128, (M, svdq.int8_ld(K))).astype(np.int8)  # the bytes past K may hold anything
    sX = (10.0 ** rng.uniform(-3, 0, M)).astype(np.float32)
    qW, sW, b = weights(N, K, M * 7 + N, bias)
    lin = svdq.Int8Linear(qW, sW, K, bias=b)
    buf = torch.full((M, N + 5), 7.0, dtype=torch.float32 if yd == "f32" else torch.bfloat16, device="cuda:0")
    Y = lin.gemm(torch.from_numpy(qX).to("cuda:0"), torch.from_numpy(sX).to("cuda:0"), ydtype, out=buf[:, :N])
    assert (buf[:, N:] == 7.0).all(), "columns past N were touched"
    check_product(Y, qX[:, :K], sX, qW[:, :K], sW, b, ydtype, f"{M}x{K}x{N} {yd}")
    Y2 = lin.gemm(torch.from_numpy(qX).to("cuda:0"), torch.from_numpy(sX).to("cuda:0"), ydtype)
    assert torch.equal(Y2, Y), "a second call differs"


def test_product_integer_extremes():
    """All codes at +-127 over the longest K: the sum 127^2 * 131072 fits 32 bits and no partial wraps."""
    torch = _torch()
    K = 131072
    for M in (2, 70):
        qX = np.full((M, K), 127, np.int8)
        qX[1::2] = -127
        qW = np.full((5, K), 127, np.int8)
        qW[2] = -127
        lin = svdq.Int8Linear(qW, np.ones(5, np.float32), K)
        Y = lin.gemm(torch.from_numpy(qX).to("cuda:0"), torch.ones(M, device="cuda:0"))
        ref = (127.0 * 127.0 * K) * np.sign(qX[:, :1].astype(float)) * np.sign(qW[:, 0].astype(float))
        np.testing.assert_array_equal(host(Y), np.float32(ref).astype(np.float64))


@pytest.mark.parametrize("M,K,N,pad", [(1, 3072, 96, 0), (4, 1000, 130, 0), (15, 320, 70, 8), (31, 129, 65, 1),
                                       (64, 3072, 128, 0), (90, 640, 200, 3), (513, 256, 300, 0)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("yd", ["f32", "gelu"])
def test_layer(M, K, N, pad, dt, yd):
    """The layer equals the quantizer and the product called one after the other, and the oracle."""
    torch = _torch()
    ydtype = {"f32": svdq.F32, "gelu": svdq.BF16_GELU}[yd]
    X = make_x(M, K, {"bf16": torch.bfloat16, "f32": torch.float32}[dt], M + K, pad)
    qW, sW, b = weights(N, K, M + N, True)
    inv = (0.2 + np.random.default_rng(N).random(K)).astype(np.float32)
    lin = svdq.Int8Linear(qW, sW, K, inv_s=inv, bias=b)
    Y = lin.forward(X, ydtype)
    assert torch.equal(Y, lin.gemm(*lin.quantize(X), ydtype))
    q, s = o8.quantize(host(X), inv)
    check_product(Y, q, s, qW[:, :K], sW, b, ydtype, f"layer {M}x{K}x{N}")


def at_any_value(shape, stride, dtype, fill, device="cuda:0"):
    """(buffer, view): a view of `shape` whose first value is the buffer's second, so that rows of an odd stride begin
    at both halves of a word; everything else of the buffer holds `fill`."""
    torch = _torch()
    span = 1 + sum((n - 1) * s for n, s in zip(shape, stride)) + 1
    buf = torch.full((span + 1,), fill, dtype=dtype, device=device)
    return buf, torch.as_strided(buf, shape, stride, 1)


@pytest.mark.parametrize("M,K,N,pad", [(1, 129, 131, 0), (4, 322, 64, 1), (70, 128, 131, 3), (300, 320, 77, 1), (90, 4609, 261, 2),
                                       (33, 2057, 40, 0), (40, 8192, 51, 2), (2, 16389, 24, 1), (4096, 301, 2051, 0), (2304, 64, 1030, 1)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("yd", ["f32", "bf16", "gelu"])
def test_rows_at_any_value(M, K, N, pad, dt, yd):
    """Rows that begin at any value, between NaNs that must not be taken in: the bits of the contiguous call, and nothing
    written beside the rows."""
    torch = _torch()
    ydtype = {"f32": svdq.F32, "bf16": svdq.BF16, "gelu": svdq.BF16_GELU}[yd]
    X = make_x(M, K, {"bf16": torch.bfloat16, "f32": torch.float32}[dt], M + K).contiguous()
    qW, sW, b = weights(N, K, M + N, True)
    lin = svdq.Int8Linear(qW, sW, K, inv_s=(0.2 + np.random.default_rng(N).random(K)).astype(np.float32), bias=b)
    want = lin.forward(X, ydtype)
    _, x = at_any_value((M, K), (K + pad, 1), X.dtype, float("nan"))
    x.copy_(X)
    buf, y = at_any_value((M, N), (N + pad, 1), want.dtype, 7.0)
    lin.forward(x, ydtype, out=y)
    assert torch.equal(y, want)
    y.fill_(7.0)
    assert (buf == 7.0).all()


def test_layer_empty_and_other_stream():
    torch = _torch()
    qW, sW, b = weights(48, 256, 3, True)
    lin = svdq.Int8Linear(qW, sW, 256, bias=b)
    assert lin.forward(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda:0")).shape == (0, 48)
    X = make_x(100, 256, torch.bfloat16, 5)
    ref = lin.forward(X)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        Y = lin.forward(X)
    s.synchronize()
    assert torch.equal(Y, ref)


def test_layer_in_a_graph():
    """The layer captured once and replayed on new inputs equals the eager calls, at few and at many tokens."""
    torch = _torch()
    qW, sW, b = weights(384, 1280, 9, True)
    lin = svdq.Int8Linear(qW, sW, 1280, bias=b)
    for M in (3, 40, 300):
        X = make_x(M, 1280, torch.bfloat16, M)
        ws, out = lin.workspace(M), torch.empty((M, 384), device="cuda:0")
        lin.forward(X, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lin.forward(X, out=out, workspace=ws)
        for k in range(4):
            X.copy_(make_x(M, 1280, torch.bfloat16, 50 + k))
            g.replay()
            torch.cuda.synchronize()
            got = out.clone()
            assert torch.equal(got, lin.forward(X)), (M, k)


def test_pack_and_forward():
    """Weights packed by the library: the layer's error against the unquantized product is that of 8 bits."""
    torch = _torch()
    from bit_diffusion_model_amd.workloads import random_layer

    wl = random_layer(200, 384, 300, 0, 11, x_out=4)
    a = svdq.act_absmax(wl.calib)
    lin = svdq.Int8Linear.from_weights(wl.W, a, 0.5)
    X = torch.from_numpy(wl.X.view(np.int16)).to("cuda:0").view(torch.bfloat16)
    ref = host(X) @ (wl.W.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    err = np.linalg.norm(host(lin.forward(X)) - ref) / np.linalg.norm(ref)
    log(f"8-bit layer against the unquantized product: {err:.2e}")
    # two roundings of step 1/127 of the row's (column's) maximum, about 4 standard deviations: 4 / 127 / sqrt(12)
    # each, doubled for the smoothed outliers that stretch some maxima
    assert err < 2 * np.sqrt(2) * 4 / 127 / np.sqrt(12)


def test_refusals():
    torch = _torch()
    qW, sW, b = weights(16, 256, 1, True)
    lin = svdq.Int8Linear(qW, sW, 256, bias=b)
    X = make_x(4, 256, torch.bfloat16, 1)
    for bad in (X[:, :255], X.half(), X.t(), X[0], X.cpu()):
        with pytest.raises(svdq.SvdqError):
            lin.forward(bad)
    with pytest.raises(svdq.SvdqError):
        lin.forward(X.expand(4, 256)[:1].expand(4, 256))  # row stride 0
    with pytest.raises(svdq.SvdqError):
        lin.forward(X, out=torch.empty((4, 17), device="cuda:0"))
    with pytest.raises(svdq.SvdqError):
        lin.forward(make_x(40, 256, torch.bfloat16, 1), workspace=torch.empty(256, dtype=torch.uint8, device="cuda:0"))
    with pytest.raises(svdq.SvdqError):
        svdq.Int8Linear(qW[:, :200].copy(), sW, 256)
    with pytest.raises(svdq.SvdqError):
        svdq.Int8Linear(qW, sW[:5], 256)
    q, s = lin.quantize(X)
    with pytest.raises(svdq.SvdqError):
        lin.gemm(q[:, :128], s)


def test_example_runs():
    """examples/spatial_block_int8.py: norm, projection, MLP and modulation together; 8 bits' error of each step."""
    import importlib.util
    import os
    import sys
    from unittest import mock

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "spatial_block_int8.py")
    spec = importlib.util.spec_from_file_location("spatial_block_int8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    with mock.patch.object(sys, "argv", ["x", "--images", "2", "--side", "12", "--channels", "320"]):
        errors = m.main()
    # per layer two roundings of at most 4 / 127 / sqrt(12) of the values' norm (maxima near 4 standard deviations),
    # doubled for smoothed outliers; the block adds three layers
    one = 2 * np.sqrt(2) * 4 / 127 / np.sqrt(12)
    assert errors["norm and projection"] < one and errors["modulation"] < one and errors["block"] < 3 * one
