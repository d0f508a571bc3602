"""GPU tests of the group norm where its output pass needs statistics of many blocks, against fp64 on the device: joined
inside (two launches), joined by a launch of their own (above 2^23 values), outputs stored past the caches (x and y above
256 MB), 256 to 2048 output blocks.  Each case says which path it is meant for.

The bound is that of test_gpu_group_norm.py with L = 128 additions in a chain: at these sizes a thread sums at most 69
positions, a group's threads meet in at most 16 + 6 additions, the blocks in at most 2 + 6 + 4; in one launch 32 values, 6
lane steps and 16 waves."""
import ctypes

import numpy as np
import pytest

from bit_diffusion_model_amd import svdq

U, L = 2.0 ** -24, 128
ACTS = {"none": svdq.GN_NONE, "silu": svdq.GN_SILU, "gelu": svdq.GN_GELU}

# (B, S, groups, C): (one launch, joined apart)
PATHS = {(2, 1000, 8, 64): (1, 0), (3, 9000, 8, 64): (0, 0), (1, 9001, 3, 9): (0, 0), (1, 5000, 3, 399): (0, 0), (2, 4096, 32, 320): (0, 0),
         (1, 70001, 4, 128): (0, 1), (1, 70001, 5, 125): (0, 1), (2, 33001, 32, 320): (0, 1)}
PAST_CACHE = [(1, 262161, 8, 128, "f32", "f32"), (1, 524321, 8, 128, "bf16", "bf16")]


def _torch():
    import torch

    return torch


@pytest.mark.parametrize("B,S,G,C", PATHS)
def test_plan(B, S, G, C):
    p = (ctypes.c_int32 * 4)()
    d = svdq._GroupNorm(C, G, 0, 1e-5, None, None)
    assert svdq.lib().svdq_debug_group_norm_plan(ctypes.byref(d), B, S, p) == 0
    assert p[0] == PATHS[B, S, G, C][0] and (p[0] or p[1] == PATHS[B, S, G, C][1])


def make(B, S, C, xd, seed, scale=1.0, offset=0.0):
    torch = _torch()
    g = torch.Generator("cuda:0").manual_seed(seed)
    x = torch.randn((B, S, C), device="cuda:0", generator=g)
    x *= scale * torch.exp(0.5 * torch.randn(C, device="cuda:0", generator=g))
    x += scale * torch.randn(C, device="cuda:0", generator=g) + offset
    gamma = 1 + 0.3 * torch.randn(C, device="cuda:0", generator=g)
    return x.to({"bf16": torch.bfloat16, "f32": torch.float32}[xd]), gamma, 0.3 * torch.randn(C, device="cuda:0", generator=g)


def reference(X, G, gamma, beta, eps, act):
    """fp64 (y, bound of its fp32 evaluation), both [B][S][C] on the device."""
    torch = _torch()
    B, S, C = X.shape
    x = X.double().reshape(B, S, G, C // G)
    mean = x.mean((1, 3), keepdim=True)
    sd = ((x - mean).square().mean((1, 3), keepdim=True) + eps).sqrt()
    z = (x - mean) / sd
    tol = 4 * L * U + L * U * z.abs() + U * (x.abs() + 2 * mean.abs()) / sd
    z, tol = z.reshape(B, S, C), tol.reshape(B, S, C)
    g, b = gamma.double(), beta.double()
    y = z * g + b
    tol = 1.13 * (g.abs() * tol + 4 * U * ((z * g).abs() + b.abs()))
    if act == "silu":
        v = y * torch.sigmoid(y)
        return v, tol + 8 * U * (1 + y.abs()) * v.abs()
    if act == "gelu":
        v = 0.5 * y * torch.special.erfc(-y * 0.5 ** 0.5)
        return v, tol + 2e-5 * v.abs()
    return y, tol


def check(Y, want, tol):
    if Y.dtype == _torch().bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    off = (Y.double() - want).abs()
    assert bool((off <= tol + 1e-37).all()), f"worst {float((off / (tol + 1e-37)).max())} of the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,G,C", PATHS)
@pytest.mark.parametrize("xd,yd,act", [("bf16", "bf16", "silu"), ("f32", "f32", "none"), ("bf16", "f32", "gelu"), ("f32", "bf16", "gelu")])
def test_group_norm(B, S, G, C, xd, yd, act):
    X, gamma, beta = make(B, S, C, xd, S + C)
    gn = svdq.GroupNorm(G, C, gamma, beta, 1e-5, ACTS[act])
    Y = gn.forward(X, svdq.F32 if yd == "f32" else svdq.BF16)
    check(Y, *reference(X, G, gamma, beta, 1e-5, act))
    assert _torch().equal(Y, gn.forward(X, svdq.F32 if yd == "f32" else svdq.BF16)), "a second call differs"


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,G,C,xd,yd", PAST_CACHE)
def test_past_the_caches(B, S, G, C, xd, yd):
    torch = _torch()
    X, gamma, beta = make(B, S, C, xd, 1)
    assert X.numel() * 2 * X.element_size() > 1 << 28
    gn = svdq.GroupNorm(G, C, gamma, beta, 1e-5, svdq.GN_SILU)
    buf = torch.full((S + 1, C), 9.0, dtype=X.dtype, device="cuda:0")
    Y = gn.forward(X, svdq.F32 if yd == "f32" else svdq.BF16, out=buf[:S][None])
    want, tol = reference(X, G, gamma, beta, 1e-5, "silu")
    check(Y, want, tol)
    assert (buf[S] == 9.0).all()
    own = X.clone()  # Y may be X itself
    gn.forward(own, svdq.F32 if yd == "f32" else svdq.BF16, out=own)
    assert torch.equal(own, Y)


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,G,C", PATHS)
@pytest.mark.parametrize("xd,act", [("bf16", "silu"), ("f32", "none"), ("bf16", "gelu")])
def test_codes(B, S, G, C, xd, act):
    """Scales within the norm's bound; codes within the half step that they stand for and the norm's bound."""
    torch = _torch()
    X, gamma, beta = make(B, S, C, xd, S)
    inv = 0.3 + torch.rand(C, device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(C))
    gn = svdq.GroupNorm(G, C, gamma, beta, 1e-5, ACTS[act])
    q, s = gn.quantize(X, inv)
    assert not q[:, C:].any()
    y, tol = reference(X, G, gamma, beta, 1e-5, act)
    f = inv.double()
    y, tol = (y * f).reshape(B * S, C), (tol * f + U * (y * f).abs()).reshape(B * S, C)
    a = y.abs().amax(1)
    s = s.double()
    assert bool(((s - a / 127).abs() <= tol.amax(1) / 127 + U * a / 127).all())
    assert bool(((q[:, :C].double() * s[:, None] - y).abs() <= s[:, None] * (0.5 + 127 * 4 * U) + tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,G,C", PATHS)
@pytest.mark.parametrize("eps", [1e-5, 1e-6, 1e-3])
def test_variance_near_eps(B, S, G, C, eps):
    """Values whose variance is about eps: another eps, or one added in another place, moves y by a fifth."""
    X, gamma, beta = make(B, S, C, "f32", S + 1, scale=0.6 * eps ** 0.5)
    Y = svdq.GroupNorm(G, C, gamma, beta, eps).forward(X, svdq.F32)
    check(Y, *reference(X, G, gamma, beta, eps, "none"))
    other, _ = reference(X, G, gamma, beta, 1.5 * eps, "none")
    assert float((Y.double() - other).abs().max()) > 0.05


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,G,C", PATHS)
def test_large_mean(B, S, G, C):
    X, gamma, beta = make(B, S, C, "f32", S + 2, offset=3000.0)
    check(svdq.GroupNorm(G, C, gamma, beta).forward(X, svdq.F32), *reference(X, G, gamma, beta, 1e-5, "none"))


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,G,C", PATHS)
def test_non_finite_groups(B, S, G, C):
    """A NaN or an infinity makes its own group of its own image NaN and no other, wherever it stands."""
    torch = _torch()
    X, gamma, beta = make(B, S, C, "f32", 3)
    cpg = C // G
    X[0, S - 1, 0] = float("nan")
    X[B - 1, S // 2, C - 1] = float("-inf")
    bad = torch.zeros((B, G), dtype=torch.bool, device="cuda:0")
    bad[0, 0] = bad[B - 1, G - 1] = True
    Y = svdq.GroupNorm(G, C, gamma, beta).forward(X, svdq.F32).view(B, S, G, cpg)
    assert torch.equal(torch.isnan(Y).all(3).all(1), bad) and torch.equal(torch.isnan(Y).any(3).any(1), bad)
    assert bool(torch.isfinite(Y).any(3).any(1)[~bad].all())


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,G,C", [k for k, v in PATHS.items() if not v[0]])
def test_other_stream_and_layout(B, S, G, C):
    """On another stream with its workspace; positions of the images interleaved ([S][B][C] seen as [B][S][C])."""
    torch = _torch()
    X, gamma, beta = make(B, S, C, "bf16", 4)
    gn = svdq.GroupNorm(G, C, gamma, beta, 1e-5, svdq.GN_SILU)
    ref, codes = gn.forward(X), gn.quantize(X)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        Y, other = gn.forward(X), gn.quantize(X)
    s.synchronize()
    assert torch.equal(Y, ref) and all(torch.equal(a, b) for a, b in zip(codes, other))
    T = X.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty((S, B, C), dtype=torch.bfloat16, device="cuda:0").transpose(0, 1)
    assert torch.equal(gn.forward(T, out=out), ref)


# Long sums: 512 blocks of statistics over inputs so large that a thread would have thousands of positions, the first of
# which (the pivot of its sums) is an outlier.  One channel to a load, so that a thread owns a single channel.
@pytest.mark.gpu
@pytest.mark.parametrize("B,S,G,C", [(512, 4096, 3, 129), (1, 1 << 20, 1, 129), (300, 9000, 1, 136)])
@pytest.mark.parametrize("sds", [3.0, 30.0, 1000.0])
def test_outliers_first(B, S, G, C, sds):
    """A thread has at most 512 positions and sums all but 8 about the mean of these 8, so that its M2 is off by at most
    512 u from the sums and 512 / 8 times 4 u from the subtraction (M2 >= 8 (pivot - mean)^2): 768 u in all."""
    torch = _torch()
    x = torch.randn((B, S, C), device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(7))
    chunk = -(-S // max(1, -(-512 // B)))  # where blocks may begin
    for at in {0, chunk, 2 * chunk, 5 * chunk, 512, 1024, S - 1}:
        if at < S:
            x[:, at] = sds
    gn = svdq.GroupNorm(G, C)
    assert gn.plan(B, S)[:2] == (0, 1)
    Y = gn.forward(x, svdq.F32)
    for b in {0, B // 2, B - 1}:
        v = x[b].double().reshape(S, G, C // G)
        mean = v.mean((0, 2), keepdim=True)
        sd = ((v - mean).square().mean((0, 2), keepdim=True) + 1e-5).sqrt()
        z = ((v - mean) / sd).reshape(S, C)
        tol = U * (768.0 * z.abs() / 2 + 4 * z.abs()) + 512 * U / 8 + U * ((v.abs() + 2 * mean.abs()) / sd).reshape(S, C)
        off = (Y[b].double() - z).abs()
        assert bool((off <= tol).all()), f"image {b}: worst {float((off / tol).max())} of the bound"
