"""Every kernel that the 8-bit product may choose, against the oracle: each case says which one it is meant for (256 compute
units), so that a choice made anew cannot leave one untested.  Sizes are ragged in M and N and end inside a stage of K;
where a block has K groups, the stages do not divide among them.

The bound is that of test_gpu_int8.py: exact integers, then at most 4 roundings and the output type's."""
import ctypes
import functools

import numpy as np
import pytest

from bit_diffusion_model_amd import svdq
from oracle import int8 as o8
from test_gpu_int8 import host, tol_product, weights

# (M, K, N): (tile, K groups, K parts, halved tiles)
VARIANTS = {
    (9, 9001, 999): (0, 1, 1, 0),
    (31, 3072, 200): (0, 1, 1, 0),
    (333, 1000, 1111): (64, 1, 1, 0),
    (501, 2100, 3001): (64, 2, 1, 0),
    (200, 5000, 1023): (64, 4, 1, 0),
    (129, 9000, 1001): (64, 4, 4, 0),
    (70, 9001, 999): (64, 4, 8, 0),
    (1497, 2050, 2101): (128, 1, 1, 0),
    (8195, 650, 643): (128, 1, 1, 0),
    (1029, 3100, 2999): (128, 2, 1, 0),
    (4090, 301, 2051): (256, 1, 1, 0),
    (4590, 1300, 3050): (256, 1, 1, 0),
    (16385, 320, 1283): (256, 1, 1, 0),
    (2500, 1000, 9301): (256, 1, 1, 114),  # the last tile row holds 196 rows: both of its halves
    (2305, 1900, 9203): (256, 1, 1, 104),  # .. 1 row: the second half is empty
}
TYPES = {"f32": svdq.F32, "bf16": svdq.BF16, "gelu": svdq.BF16_GELU}


@pytest.mark.parametrize("M,K,N", VARIANTS)
def test_plan(M, K, N):
    """The choice at 256 compute units (what the library assumes on a host without a GPU)."""
    p = (ctypes.c_int32 * 4)()
    lay = svdq._Int8Layer(K, N, None, 16, 16, None)
    assert svdq.lib().svdq_debug_w8a8_plan(ctypes.byref(lay), M, p) == 0
    assert tuple(p) == VARIANTS[M, K, N]


def test_plan_refusals():
    L, p = svdq.lib(), (ctypes.c_int32 * 4)()
    lay = svdq._Int8Layer(64, 64, None, 16, 16, None)
    assert L.svdq_debug_w8a8_plan(ctypes.byref(lay), 0, p) == 1 and L.svdq_debug_w8a8_plan(None, 4, p) == 1
    assert L.svdq_debug_w8a8_plan(ctypes.byref(lay), 4, None) == 1 and L.svdq_debug_w8a8_plan(ctypes.byref(lay), 1 << 30, p) == 2
    nrm = svdq._GroupNorm(64, 8, 0, 1e-5, None, None)
    assert L.svdq_debug_group_norm_plan(ctypes.byref(nrm), 0, 4, p) == 1 and L.svdq_debug_group_norm_plan(None, 1, 4, p) == 1
    assert L.svdq_debug_group_norm_plan(ctypes.byref(nrm), 1, 4, None) == 1
    assert L.svdq_debug_group_norm_plan(ctypes.byref(nrm), 70000, 4, p) == 2


@functools.lru_cache(maxsize=1)
def problem(M, K, N):
    rng = np.random.default_rng(M + K + N)
    qX = rng.integers(-127, 128, (M, svdq.int8_ld(K))).astype(np.int8)  # the bytes past K may hold anything
    sX = (10.0 ** rng.uniform(-3, 0, M)).astype(np.float32)
    sX[M // 3] = np.nan  # a row that held a NaN
    qW, sW, b = weights(N, K, M * 7 + N, True)
    # values near 1, where GELU bends: the sums are about 73^2 sqrt(K)
    sW *= np.float32(1.0 / (73.0 * 73.0 * np.sqrt(K) * 1e-2))
    return qX, sX, qW, sW, b, o8.product(qX[:, :K], sX, qW[:, :K], sW)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", VARIANTS)
@pytest.mark.parametrize("yd", TYPES)
@pytest.mark.parametrize("bias", [True, False])
def test_product(M, K, N, yd, bias):
    import torch

    qX, sX, qW, sW, b, p = problem(M, K, N)
    b = b if bias else None
    lin = svdq.Int8Linear(qW, sW, K, bias=b)
    assert lin.plan(M) == VARIANTS[M, K, N]
    buf = torch.full((M + 1, N + 5), 7.0, dtype=torch.float32 if yd == "f32" else torch.bfloat16, device="cuda:0")
    x, s = torch.from_numpy(qX).to("cuda:0"), torch.from_numpy(sX).to("cuda:0")
    Y = lin.gemm(x, s, TYPES[yd], out=buf[:M, :N])
    assert (buf[:, N:] == 7.0).all() and (buf[M] == 7.0).all(), "values past M or N were touched"
    ref = p if b is None else p + b
    ref = o8.gelu(ref) if yd == "gelu" else ref
    tol = np.broadcast_to(tol_product(p, b, TYPES[yd]), ref.shape)
    got, nan = host(Y), np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan) and nan[M // 3].all()
    err = np.abs(got - ref)
    err[nan] = 0.0
    worst = np.max(err / np.where(nan, 1.0, tol))
    assert worst <= 1.0, f"{worst} of the bound"
    assert torch.equal(torch.nan_to_num(lin.gemm(x, s, TYPES[yd])), torch.nan_to_num(Y)), "a second call differs"


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(2500, 1000, 9301), (1029, 3100, 2999), (501, 2100, 3001), (129, 9000, 1001)])
def test_layer(M, K, N):
    """The layer on odd rows equals the quantizer and the product, whose codes are the oracle's."""
    import torch

    rng = np.random.default_rng(K)
    qW, sW, b = weights(N, K, 5, True)
    inv = (0.2 + rng.random(K)).astype(np.float32)
    lin = svdq.Int8Linear(qW, sW, K, inv_s=inv, bias=b)
    X = torch.randn((M, K + 1), device="cuda:0").to(torch.bfloat16)[:, :K]
    q, s = lin.quantize(X)
    qo, so = o8.quantize(host(X), inv)
    assert np.array_equal(q.cpu().numpy()[:, :K], qo) and np.array_equal(s.cpu().numpy(), so)
    assert torch.equal(lin.forward(X, svdq.BF16_GELU), lin.gemm(q, s, svdq.BF16_GELU))
