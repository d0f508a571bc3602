"""Every kernel that the block-scaled product and the layer norm may choose, against the oracle: each case says which one it
is meant for (256 compute units), so that a choice made anew cannot leave one untested.  Sizes are ragged in M and N and
end inside a block of K or a chunk of a row.  Bounds as in test_gpu_fp8.py and test_gpu_layer_norm.py."""
import ctypes
import functools

import numpy as np
import pytest

from bit_diffusion_model_amd import svdq
from oracle import fp8 as o

# (M, K, N): plans for fp32 and for bf16 outputs: (rows and columns of a tile, K groups, K parts)
VARIANTS = {
    (9, 9001, 999): ((0, 16, 1, 1), (0, 16, 1, 1)),
    (31, 2944, 200): ((0, 16, 1, 1), (0, 16, 1, 1)),
    (333, 1000, 1111): ((64, 64, 1, 1), (64, 64, 1, 1)),
    (501, 2100, 3001): ((64, 64, 1, 1), (64, 64, 2, 1)),
    (32, 3000, 18432): ((64, 64, 2, 1), (64, 64, 2, 1)),
    (200, 5000, 1023): ((64, 64, 4, 4), (64, 64, 4, 1)),
    (70, 9001, 999): ((64, 64, 4, 8), (64, 64, 4, 8)),
    (1029, 3100, 2999): ((128, 128, 2, 1), (128, 128, 2, 1)),
    (8195, 650, 643): ((64, 64, 1, 1), (128, 128, 1, 1)),
    (2500, 1000, 9301): ((128, 128, 1, 1), (128, 128, 1, 1)),
    (4090, 301, 2051): ((64, 64, 1, 1), (192, 256, 1, 1)),
    (2305, 1900, 9203): ((128, 128, 1, 1), (192, 256, 1, 1)),  # the last tile row holds 1 row
    (2323, 1483, 5205): ((64, 64, 1, 1), (224, 256, 1, 1)),  # .. 83: four of its waves none
    (4701, 2196, 2601): ((64, 64, 1, 1), (224, 256, 1, 1)),  # .. 221: its last wave half full
    (2685, 1299, 5584): ((128, 128, 1, 1), (256, 256, 1, 1)),
    (4090, 600, 4090): ((128, 128, 1, 1), (256, 256, 1, 1)),
}
TYPES = {"f32": svdq.F32, "bf16": svdq.BF16, "gelu": svdq.BF16_GELU}

# (B, S, C): (lanes, chunks, waves to a row, blocks of the gradient; negative: columns to a block of their own)
NORMS = {
    (1, 5, 8): (16, 1, 1, -16), (1, 2000, 33): (16, 1, 1, 16), (2, 1500, 64): (16, 1, 1, 24), (1, 3000, 65): (16, 1, 1, 47),
    (1, 5, 100): (16, 1, 1, -16), (1, 5, 200): (32, 1, 1, -16), (1, 5, 700): (64, 1, 2, -16), (1, 5, 2041): (64, 1, 4, -16),
    (1, 5, 3001): (64, 2, 3, -32), (1, 5, 8001): (64, 2, 8, -64), (1, 5, 9000): (64, 4, 5, -64), (1, 5, 16383): (64, 4, 8, 5),
    (1, 1023, 100): (16, 1, 1, -16), (1, 999, 1111): (64, 3, 1, -16), (2, 450, 2047): (64, 4, 1, -16), (1, 1000, 5003): (64, 2, 5, -64),
    (1, 5000, 100): (16, 1, 1, 79), (1, 5000, 250): (16, 2, 1, 157), (1, 5000, 300): (16, 3, 1, 157),
    (1, 5000, 500): (16, 4, 1, 157), (1, 5000, 700): (32, 3, 1, 209), (1, 5000, 1000): (32, 4, 1, 209),
    (1, 3000, 1300): (64, 3, 1, 200), (2, 1500, 2047): (64, 4, 1, 250), (1, 2100, 3001): (64, 3, 2, 210),
    (1, 1100, 5003): (64, 2, 5, 220), (1, 600, 9001): (64, 3, 6, -64), (1, 1050, 9001): (64, 3, 6, 210),
    (1, 300, 16383): (64, 4, 8, 150),
}


@pytest.mark.parametrize("M,K,N", VARIANTS)
def test_plan(M, K, N):
    """The choice at 256 compute units (what the library assumes on a host without a GPU)."""
    p = (ctypes.c_int32 * 4)()
    lay = svdq._Fp8Layer(K, N, 16, 16, None)
    for yd in (svdq.F32, svdq.BF16):
        assert svdq.lib().svdq_debug_fp8_plan(ctypes.byref(lay), M, yd, p) == 0
        assert tuple(p) == VARIANTS[M, K, N][yd]


@pytest.mark.parametrize("B,S,C", NORMS)
def test_norm_plan(B, S, C):
    p = (ctypes.c_int32 * 4)()
    n = svdq._LayerNorm(C, 1e-5, 0, None, None, 0)
    assert svdq.lib().svdq_debug_layer_norm_plan(ctypes.byref(n), B, S, p) == 0
    assert tuple(p) == NORMS[B, S, C]


def test_every_row_has_its_lanes():
    """Whatever the sizes: the lanes cover a row and its codes up to a multiple of 128, all chunks but a lane's last two (16
    and 32 lanes: but the last) lie within the row, and every wave holds a part of it."""
    p, L = (ctypes.c_int32 * 4)(), svdq.lib()
    for C in [*range(1, 2000), *range(2001, 16385, 37), 16384]:
        n = svdq._LayerNorm(C, 1e-5, 0, None, None, 0)
        for rows in (1, 300, 1500, 5000, 100000):
            assert L.svdq_debug_layer_norm_plan(ctypes.byref(n), 1, rows, p) == 0
            lanes, chunks, waves, _ = p
            step = 8 * lanes * waves
            assert step * chunks >= svdq.int8_ld(C) and 1 <= waves <= 16 and 512 * (waves - 1) < C
            assert (chunks - (2 if lanes == 64 else 1)) * step <= C
            assert waves <= {1: 4, 2: 13, 3: 10, 4: 8}[chunks]  # what the kernels are compiled for


def test_plan_refusals():
    L, p = svdq.lib(), (ctypes.c_int32 * 4)()
    lay = svdq._Fp8Layer(64, 64, 16, 16, None)
    assert L.svdq_debug_fp8_plan(ctypes.byref(lay), 0, 0, p) == 1 and L.svdq_debug_fp8_plan(None, 4, 0, p) == 1
    assert L.svdq_debug_fp8_plan(ctypes.byref(lay), 4, 0, None) == 1 and L.svdq_debug_fp8_plan(ctypes.byref(lay), 1 << 30, 0, p) == 2
    n = svdq._LayerNorm(64, 1e-5, 0, None, None, 0)
    assert L.svdq_debug_layer_norm_plan(ctypes.byref(n), 0, 4, p) == 1 and L.svdq_debug_layer_norm_plan(None, 1, 4, p) == 1
    assert L.svdq_debug_layer_norm_plan(ctypes.byref(n), 1, 4, None) == 1
    assert L.svdq_debug_layer_norm_plan(ctypes.byref(n), 70000, 4, p) == 2


@functools.lru_cache(maxsize=1)
def problem(M, K, N):
    from test_gpu_fp8 import weights

    qX, _, _ = weights(M, K, M + K + N)
    sX = (10.0 ** np.random.default_rng(M).uniform(-3, 0, (o.blocks(K), svdq.fp8_scale_ld(M)))).astype(np.float32)
    sX[:, M:] = np.nan
    sX[-1, M // 3] = np.nan  # a row whose last block held a NaN
    qW, sW, b = weights(N, K, M * 7 + N)
    sW *= np.float32(1e-5)  # values near 1, where GELU bends
    return qX, sX, qW, sW, b * np.float32(1e-2)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", VARIANTS)
@pytest.mark.parametrize("yd", TYPES)
def test_product(M, K, N, yd):
    import torch

    from test_gpu_fp8 import check, dev, fp8_dev

    qX, sX, qW, sW, b = problem(M, K, N)
    for bias in (b, None):
        lin = svdq.Fp8Linear(qW, sW, K, bias=bias)
        assert lin.plan(M, TYPES[yd]) == VARIANTS[M, K, N][0 if yd == "f32" else 1]
        buf = torch.full((M + 1, N + 5), 7.0, dtype=torch.float32 if yd == "f32" else torch.bfloat16, device="cuda:0")
        x, s = fp8_dev(qX), dev(sX)
        Y = lin.gemm(x, s, TYPES[yd], out=buf[:M, :N])
        assert (buf[:, N:] == 7.0).all() and (buf[M] == 7.0).all(), "values past M or N were touched"
        assert Y[M // 3].isnan().all()
        check(Y, qX, sX, qW, sW, bias, TYPES[yd], f"{M}x{K}x{N} {yd}")
        assert torch.equal(torch.nan_to_num(lin.gemm(x, s, TYPES[yd])), torch.nan_to_num(Y)), "a second call differs"


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,C", NORMS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 1])
def test_norm(B, S, C, dt, pad):
    """The norm, its codes and its gradient on each way to hold a row; rows beside each other and at odd places."""
    import torch

    from test_gpu_fp8 import codes
    from test_gpu_layer_norm import check_norm, make, params

    X = make(B, S, C, dt, B + S + C, pad)
    g, b = params(B, C, False, C)
    ln = svdq.LayerNorm(C, g, b, 1e-5)
    assert ln.plan(B, S) == NORMS[B, S, C]
    stats = ln.alloc_stats(X)
    Y = ln.forward(X, svdq.F32, stats=stats)
    check_norm(Y, X, g, b, False, 1e-5, False, stats, f"{B}x{S}x{C}")
    q, s = ln.quantize(X)
    q2, s2 = svdq.quantize_act_fp8(Y.view(B * S, C))
    assert torch.equal(s[:, :B * S], s2[:, :B * S]) and np.array_equal(codes(q), codes(q2))
    dY = make(B, S, C, dt, C + 1, pad)
    dX, dg, db = ln.backward(dY, X, stats)
    z = (X.double() - stats[0].double().view(B, S, 1)) * stats[1].double().view(B, S, 1)
    for got, t in ((dg, dY.double() * z), (db, dY.double())):
        bound = 2.0 ** -24 * (B * S + 6) * t.abs().sum((0, 1)) + 1e-37
        assert ((got.double() - t.sum((0, 1))).abs() <= bound).all()
    w = torch.from_numpy(g).cuda().double()
    gg = dY.double() * w
    ref = (gg - gg.mean(2, keepdim=True) - z * (gg * z).mean(2, keepdim=True)) * stats[1].double().view(B, S, 1)
    u = 2.0 ** -24
    tol = stats[1].double().view(B, S, 1) * u * (6 * gg.abs() + 50 * gg.abs().mean(2, keepdim=True)
                                                 + 54 * z.abs() * (gg * z).abs().mean(2, keepdim=True)) + 3 * u * ref.abs() + 1e-37
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * ref.abs()
    assert ((dX.double() - ref).abs() <= tol).all()
    # in place: the sums by the blocks of rows
    out = dY.contiguous().clone()
    dX2, dg2, db2 = ln.backward(out, X, stats, out=out)
    assert dX2 is out and torch.equal(dX2, dX)
    for got, t in ((dg2, dY.double() * z), (db2, dY.double())):
        bound = 2.0 ** -24 * (B * S + 6) * t.abs().sum((0, 1)) + 1e-37
        assert ((got.double() - t.sum((0, 1))).abs() <= bound).all()
