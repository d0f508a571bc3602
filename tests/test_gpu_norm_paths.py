"""GPU tests of the group norm on each of its paths: one launch (no workspace), statistics and output in two launches,
and three launches (the blocks' statistics joined by a launch of their own, above 2^23 values)."""
import numpy as np
import pytest

from bit_diffusion_model_amd import svdq
from test_gpu_int8 import host

pytestmark = pytest.mark.gpu


def _torch():
    import torch

    return torch


# (B, S, groups, C, whether one launch serves it): vectors of 8, 4, 2 and 1 channels, groups of 1 to 40 channels
CONSTANT = [(2, 1024, 32, 640, True), (1, 2048, 4, 64, True), (2, 64, 32, 1280, True), (1, 1000, 5, 15, True), (1, 700, 7, 42, True),
            (1, 1, 4, 64, True), (2, 6000, 8, 64, False), (1, 9001, 3, 9, False), (1, 70001, 4, 128, False)]


@pytest.mark.parametrize("B,S,G,C,one", CONSTANT)
@pytest.mark.parametrize("value", [0.1, 100.1, 1000.1, 3000.7, -33333.3])
def test_constant_group_gives_beta(B, S, G, C, one, value):
    """A group of one value: its mean is that value and x - mean is 0, whatever the value, so y is beta to the bit.
    (Sums of such values are not exact in fp32: a mean that is off by one bit of 3000.7 moves y by 0.08 at eps = 1e-5.)
    The other groups hold normals around the value."""
    torch = _torch()
    rng = np.random.default_rng(S + C)
    x = (rng.standard_normal((B, S, C)) + value).astype(np.float32)
    cpg = C // G
    x[:, :, :cpg] = np.float32(value)
    x[B - 1, :, C - cpg:] = np.float32(value)
    X = torch.from_numpy(x).to("cuda:0")
    beta = (0.3 * rng.standard_normal(C)).astype(np.float32)
    gn = svdq.GroupNorm(G, C, (1 + 0.3 * rng.standard_normal(C)).astype(np.float32), beta)
    assert (gn.workspace(B, S, X.device) is None) == one
    Y = host(gn.forward(X, svdq.F32))
    want = beta.astype(np.float64)
    assert np.array_equal(Y[:, :, :cpg], np.broadcast_to(want[:cpg], (B, S, cpg)))
    assert np.array_equal(Y[B - 1, :, C - cpg:], np.broadcast_to(want[C - cpg:], (S, cpg)))


@pytest.mark.parametrize("B,S,C", [(2, 1024, 640), (2, 64, 1280), (1, 2000, 24), (1, 9001, 64)])
def test_constant_image_gives_zero_codes(B, S, C):
    """Without gamma and beta an image of one value is 0 everywhere: codes 0 and the smallest scale."""
    torch = _torch()
    X = torch.full((B, S, C), 3000.7, device="cuda:0")
    q, s = svdq.GroupNorm(8, C).quantize(X)
    assert not q.any() and torch.equal(s, torch.full_like(s, float(np.float32(2.0 ** -96) / np.float32(127))))


@pytest.mark.parametrize("B,S,G,C,one", [(3, 150, 8, 96, True), (2, 6000, 8, 64, False), (1, 5003, 3, 9, False), (1, 5000, 8, 264, False),
                                         (1, 70001, 4, 128, False)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 3])
def test_in_place(B, S, G, C, one, xd, pad):
    """Y may be X itself, on every path: the bits of the call into another tensor."""
    torch = _torch()
    buf = torch.randn((B, S, C + pad), device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(C))
    buf = buf.to({"bf16": torch.bfloat16, "f32": torch.float32}[xd])
    X, rest = buf[:, :, :C], buf[:, :, C:].clone()
    gn = svdq.GroupNorm(G, C, act=svdq.GN_SILU)
    assert (gn.workspace(B, S, X.device) is None) == one
    ydtype = svdq.F32 if xd == "f32" else svdq.BF16
    want = gn.forward(X, ydtype)
    assert gn.forward(X, ydtype, out=X) is X
    assert torch.equal(X, want) and torch.equal(buf[:, :, C:], rest)


@pytest.mark.parametrize("B,S,G,C", [(3, 64, 8, 96), (2, 6000, 8, 64), (5, 41, 3, 33), (2, 40000, 4, 128)])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_one_image_as_many(B, S, G, C, xd):
    """An image expanded over the batch (image stride 0) gives the bits of its copies; only Y's images have to be apart."""
    torch = _torch()
    one = torch.randn((1, S, C), device="cuda:0", generator=torch.Generator("cuda:0").manual_seed(S))
    one = one.to({"bf16": torch.bfloat16, "f32": torch.float32}[xd])
    X, copies = one.expand(B, S, C), one.repeat(B, 1, 1)
    gn = svdq.GroupNorm(G, C, act=svdq.GN_SILU)
    assert torch.equal(gn.forward(X, svdq.F32), gn.forward(copies, svdq.F32))
    for a, b in zip(gn.quantize(X), gn.quantize(copies)):
        assert torch.equal(a, b)
    lin = svdq.Int8Linear(np.ones((20, svdq.int8_ld(C)), np.int8), np.ones(20, np.float32), C)
    assert torch.equal(gn.forward_linear(X, lin), gn.forward_linear(copies, lin))
    with pytest.raises(svdq.SvdqError, match="bsy"):
        gn.forward(X, svdq.F32 if xd == "f32" else svdq.BF16, out=X)
