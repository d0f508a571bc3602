"""The layer norm and the block quantizer where a call takes several launches (2^21 workgroups each; the quantizer 2^24 - 1),
and rows held by the widest teams of waves.  A row's result does not depend on its place, so the rows of the later
launches are held against the same rows run alone, to the bit."""
import ctypes

import numpy as np
import pytest

from bit_diffusion_model_amd import svdq

# C: (lanes, chunks, waves) of a row, at as many rows as the card likes
TEAMS = {13001: (64, 2, 13), 12289: (64, 2, 13), 13312: (64, 2, 13), 15001: (64, 3, 10), 14337: (64, 3, 10)}


@pytest.mark.parametrize("C", TEAMS)
def test_plan_of_wide_teams(C):
    p = (ctypes.c_int32 * 4)()
    n = svdq._LayerNorm(C, 1e-5, 0, None, None, 0)
    assert svdq.lib().svdq_debug_layer_norm_plan(ctypes.byref(n), 1, 200, p) == 0
    assert tuple(p)[:3] == TEAMS[C]


@pytest.mark.gpu
@pytest.mark.parametrize("C", TEAMS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 1])
def test_wide_teams(C, dt, pad):
    import torch

    from test_gpu_fp8 import codes
    from test_gpu_layer_norm import check_norm, make, params

    B, S = 2, 100
    X = make(B, S, C, dt, C, pad)
    X[1, 7, C - 1] = float("nan")
    g, b = params(B, C, True, C)
    ln = svdq.LayerNorm(C, g, b, 1e-5, one_plus=True)
    assert ln.plan(B, S)[:3] == TEAMS[C]
    stats = ln.alloc_stats(X)
    Y = ln.forward(X, svdq.F32, stats=stats)
    assert Y[1, 7].isnan().all() and Y.isnan().sum() == C
    q, s = ln.quantize(X)
    q2, s2 = svdq.quantize_act_fp8(Y.view(B * S, C))
    M = B * S
    assert torch.equal(s[:, :M].nan_to_num(-1.0), s2[:, :M].nan_to_num(-1.0)) and np.array_equal(codes(q), codes(q2))
    X[1, 7, C - 1], clean = 0.0, Y.clone()
    Z = ln.forward(X, svdq.F32, stats=stats)
    check_norm(Z, X, g, b, True, 1e-5, True, stats, f"{C}")
    clean[1, 7] = Z[1, 7]
    assert torch.equal(Z, clean)


@pytest.mark.gpu
@pytest.mark.parametrize("S,B,C,waves", [(1 << 20, 32, 8, 1), (1 << 17, 64, 1025, 1), (1 << 16, 32, 4097, 3)])
def test_norm_of_several_launches(S, B, C, waves):
    """One image B times and a few of its rows more (image stride 0), which is a launch's rows and some; the last image's
    rows are the first one's."""
    import torch

    torch.manual_seed(C)
    X = torch.randn(1, S, C, device="cuda:0").bfloat16()
    ln = svdq.LayerNorm(C, 1 + 0.3 * torch.randn(C, device="cuda:0"), torch.randn(C, device="cuda:0"))
    rows = B * S  # of one launch: 2^21 workgroups of 16 rows (16 lanes each), 4 (a wave each) or 1
    assert rows == (1 << 21) * (16 if C <= 128 else 4 if waves == 1 else 1) and ln.plan(B + 1, S)[2] == waves
    want, stats = torch.empty_like(X), ln.alloc_stats(X)
    ln.forward(X, out=want, stats=stats)
    many = X.expand(B + 1, S, C)
    out, st = torch.full((B + 1, S, C), 7.0, dtype=X.dtype, device="cuda:0"), torch.full((2, rows + S), 7.0, device="cuda:0").unbind()
    ln.forward(many, out=out, stats=st)
    for i in range(B + 1):
        assert torch.equal(out[i], want[0]), i
        assert all(torch.equal(a[i * S:i * S + S], w) for a, w in zip(st, stats)), i


@pytest.mark.gpu
def test_codes_of_several_launches():
    """The norm into codes and the quantizer, 8 values a row, beyond a launch's rows: codes, scales and what is not a row."""
    import torch

    torch.manual_seed(0)
    C = 8
    for rows, most in (((1 << 25) + 37, 1 << 25), (4 * ((1 << 24) - 1) + 37, 4 * ((1 << 24) - 1))):
        X = torch.randn(rows, C, device="cuda:0").bfloat16()
        ln = svdq.LayerNorm(C)
        make = ln.quantize if most == 1 << 25 else svdq.quantize_act_fp8
        q = torch.full((rows + 1, 128), 7, dtype=torch.uint8, device="cuda:0")
        s = torch.full((1, svdq.fp8_scale_ld(rows)), 7.0, device="cuda:0")
        make(X, out=(q[:rows].view(torch.float8_e4m3fn), s))
        assert (q[rows] == 7).all() and (s[0, rows:] == 7.0).all()
        for a, b in ((0, 1000), (most - 1000, most), (most, rows), (most - 3, most + 3)):
            qa, sa = make(X[a:b])
            assert torch.equal(q[a:b], qa.view(torch.uint8)) and torch.equal(s[0, a:b], sa[0, :b - a]), (a, b)
        del q, s, X
