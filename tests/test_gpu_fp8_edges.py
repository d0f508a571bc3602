"""Calls of the layer norm's gradient and the block-scaled product that other tests do not make: rows far apart, images that
do not follow each other, one image for all, NaN and infinities in the gradient, two streams at once.  Results are held
against the same call on rows side by side: a row's arithmetic does not depend on where it lies, so dX is the same to the
bit, and the columns' sums of one kernel are too; those of another order are within 2^-24 (rows + 6) of the magnitudes."""
import ctypes

import numpy as np
import pytest

from bit_diffusion_model_amd import svdq

EINVAL = 1


def test_eps_is_a_normal_number():
    L, p = svdq.lib(), (ctypes.c_int32 * 4)()
    for eps, want in ((1.17549435e-38, 0), (1.1e-38, EINVAL), (1e-45, EINVAL), (float("inf"), EINVAL), (-1e-5, EINVAL)):
        n = svdq._LayerNorm(64, eps, 0, None, None, 0)
        assert L.svdq_debug_layer_norm_plan(ctypes.byref(n), 1, 4, p) == want


def setup(B, S, C, dt, modulated, seed=0):
    import torch

    torch.manual_seed(seed)
    t = dict(f32=torch.float32, bf16=torch.bfloat16)[dt]
    x, dy = (torch.randn(B, S, C, device="cuda:0").to(t) for _ in range(2))
    shape = (B, C) if modulated else (C,)
    ln = svdq.LayerNorm(C, 1 + 0.3 * torch.randn(*shape, device="cuda:0"), torch.randn(*shape, device="cuda:0"))
    stats = ln.alloc_stats(x)
    ln.forward(x, stats=stats)
    return x, dy, ln, stats


def sums_close(ln, got, want, x, dy, stats):
    m, r = (t.double().view(*x.shape[:2], 1) for t in stats)
    z = (x.double() - m) * r
    dims = (1,) if ln.images else (0, 1)
    rows = x.shape[1] if ln.images else x.shape[0] * x.shape[1]
    for a, b, t in zip(got, want, (dy.double() * z, dy.double())):
        assert ((a.double() - b.double()).abs() <= 2 * 2.0 ** -24 * (rows + 6) * t.abs().sum(dims) + 1e-37).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,C", [(3, 40, 200), (2, 333, 1111), (5, 1, 96), (2, 7, 9000)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("modulated", [False, True])
def test_gradient_of_images_apart(B, S, C, dt, modulated):
    import torch

    x, dy, ln, stats = setup(B, S, C, dt, modulated)
    want = ln.backward(dy, x, stats)
    wide = torch.full((B, S + 3, C + 5), float("nan"), dtype=x.dtype, device=x.device)
    for kind in ("x", "dy", "both"):
        xs, ds = x, dy
        if kind != "dy":
            xs = wide.clone()[:, :S, :C]
            xs.copy_(x)
        if kind != "x":
            ds = wide.clone()[:, 1:S + 1, 2:C + 2]
            ds.copy_(dy)
        got = ln.backward(ds, xs, stats)
        assert torch.equal(got[0], want[0]), kind
        sums_close(ln, got[1:], want[1:], x, dy, stats)


@pytest.mark.gpu
@pytest.mark.parametrize("modulated", [False, True])
def test_gradient_of_one_image_for_all(modulated):
    import torch

    B, S, C = 4, 30, 320
    x, dy, ln, stats = setup(B, S, C, "f32", modulated)
    one = x[:1].expand(B, S, C)
    ln.forward(one.contiguous(), stats=stats)
    want = ln.backward(dy, one.contiguous(), stats)
    got = ln.backward(dy, one, stats)
    assert torch.equal(got[0], want[0])
    sums_close(ln, got[1:], want[1:], one, dy, stats)


@pytest.mark.gpu
@pytest.mark.parametrize("S,stride", [(2, (1 << 28) - 64), (3, 1 << 28)])
def test_gradient_of_rows_far_apart(S, stride):
    """A run whose rows lie within 2 GB is read at 32-bit offsets, a longer one is not."""
    import torch

    C = 700
    x, dy, ln, stats = setup(1, S, C, "f32", False)
    want = ln.backward(dy, x, stats)
    buf = torch.empty((S - 1) * stride + C, device="cuda:0")
    far = buf.as_strided((1, S, C), (0, stride, 1))
    far.copy_(x)
    got = ln.backward(dy, far, stats)
    assert torch.equal(got[0], want[0])
    sums_close(ln, got[1:], want[1:], x, dy, stats)
    far.copy_(dy)
    got = ln.backward(far, x, stats)
    assert torch.equal(got[0], want[0])
    sums_close(ln, got[1:], want[1:], x, dy, stats)


@pytest.mark.gpu
@pytest.mark.parametrize("S", [5, 400, 1500])
def test_gradient_of_nan_and_infinite_values(S):
    """In x: its row of dX and, since it is a term of them, all of dgamma.  In dy: its row and its column of the sums."""
    import torch

    C = 333
    for place in ("x", "dy"):
        x, dy, ln, stats = setup(1, S, C, "f32", False)
        (x if place == "x" else dy)[0, S // 2, 17] = float("nan") if S != 400 else float("inf")
        ln.forward(x, stats=stats)
        own = dy.clone()
        for out in (None, own):  # the columns by blocks of their own, and by the blocks of rows
            dx, dg, db = ln.backward(own, x, stats, out=out)
            bad = ~dx.isfinite()[0]
            assert bad[S // 2].all() and not bad[:S // 2].any() and not bad[S // 2 + 1:].any()
            if place == "x":
                assert dg.isnan().all() and db.isfinite().all()
            else:
                only = torch.arange(C, device="cuda:0") == 17
                assert torch.equal(~dg.isfinite(), only) and torch.equal(~db.isfinite(), only)


@pytest.mark.gpu
@pytest.mark.parametrize("S", [77, 999, 3000])
def test_gradients_on_two_streams_at_once(S):
    import torch

    sets = [setup(2, S, 1024, "bf16", True, seed) for seed in (1, 2)]
    want = [ln.backward(dy, x, stats) for x, dy, ln, stats in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, (x, dy, ln, stats) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(ln.backward(dy, x, stats))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.gpu
@pytest.mark.parametrize("S", [16, 700])
def test_gradient_captured_and_replayed(S):
    """A captured gradient on new inputs, with other calls between the replays."""
    import torch

    x, dy, ln, stats = setup(2, S, 500, "f32", False)
    sets = [setup(2, S, 500, "f32", False, seed)[:2] for seed in (3, 4, 5)]
    ln.backward(dy, x, stats)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ln.forward(x, svdq.F32, stats=stats)
        out = ln.backward(dy, x, stats)
    for a, b in sets + sets[:1]:
        x.copy_(a)
        dy.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        other = ln.alloc_stats(a)
        ln.forward(a, svdq.F32, stats=other)
        want = ln.backward(b, a, other)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(223, 256, 20000), (224, 130, 29000), (225, 384, 29000), (193, 256, 33000), (2240, 128, 2560)])
def test_product_rows_do_not_depend_on_their_tile(M, K, N):
    """A row's sums run over K alone and in one order: the first rows of a product are those of a smaller one wherever both
    run without K groups, and a row of codes beside a NaN scale is not touched by it."""
    import torch

    torch.manual_seed(M)
    q = (torch.randn(N, svdq.int8_ld(K), device="cuda:0") * 40).to(torch.float8_e4m3fn)
    q.view(torch.uint8)[:, K:] = 0
    sW = torch.rand(svdq.fp8_blocks(N), svdq.fp8_blocks(K), device="cuda:0") * 1e-3
    lin = svdq.Fp8Linear(q, sW, K)
    x = torch.randn(M, K, device="cuda:0")
    x[M - 1, 0] = float("nan")
    qX, sX = svdq.quantize_act_fp8(x)
    Y = lin.gemm(qX, sX, svdq.BF16)
    rows, groups = lin.plan(M, svdq.BF16)[0], lin.plan(M, svdq.BF16)[2]
    assert rows >= 64 and groups == 1
    assert Y[M - 1].isnan().all() and Y[:M - 1].isfinite().all()
    half = M // 2
    part = lin.gemm(*svdq.quantize_act_fp8(x[:half].contiguous()), svdq.BF16)
    assert lin.plan(half, svdq.BF16)[2] == 1 and torch.equal(part, Y[:half])
    assert np.isfinite(float(Y[:M - 1].float().abs().max()))
