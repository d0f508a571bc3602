"""A row that holds a NaN has a NaN scale and zero codes, whatever the NaN's bits: no call writes a payload as a code."""
import numpy as np
import pytest

from bit_diffusion_model_amd import svdq

pytestmark = pytest.mark.gpu
# quiet and signalling NaNs of both signs with every byte of the payload set somewhere
NANS = [0x7FC00000, 0x7FC00001, 0xFFC123A5, 0x7F8000FF, 0xFF800080, 0x7FFFFFFF, 0xFFFFFFFF]


def _torch():
    import torch

    return torch


def nan_rows(K):
    """[len(NANS) + 2][K] normals: row i + 1 holds NANS[i], the last row an infinity, row 0 only numbers."""
    x = np.random.default_rng(K).standard_normal((len(NANS) + 2, K)).astype(np.float32)
    for i, bits in enumerate(NANS):
        x.view(np.uint32)[i + 1, (7 * i + 3) % K] = bits
    x[-1, K // 2] = -np.inf
    return x


# one and four waves per row, rows in registers and read twice
@pytest.mark.parametrize("K", [1, 40, 300, 1000, 2048, 5000, 16384, 16500])
@pytest.mark.parametrize("smooth", [False, True])
def test_quantizer(K, smooth):
    torch = _torch()
    X = torch.from_numpy(nan_rows(K)).to("cuda:0")
    q, s = svdq.quantize_act_int8(X, torch.full((K,), 0.7, device="cuda:0") if smooth else None)
    assert torch.isnan(s[1:]).all() and torch.isfinite(s[0])
    assert not q[1:].any() and q[0].any()


@pytest.mark.parametrize("bits", [0x7FC0, 0x7F81, 0xFFFF, 0xFF80])
def test_quantizer_bf16(bits):
    torch = _torch()
    x = np.full((2, 320), 0x3F80, np.uint16)
    x[1, 17] = bits
    q, s = svdq.quantize_act_int8(torch.from_numpy(x.view(np.int16)).to("cuda:0").view(torch.bfloat16))
    assert torch.isnan(s[1]) and not q[1].any() and (q[0, :320] == 127).all()  # zeros past the row's values


def test_quantizer_nan_smoothing():
    """A NaN in the smoothing factors reaches every row."""
    torch = _torch()
    inv = np.ones(320, np.float32)
    inv.view(np.uint32)[5] = 0x7FC000FF
    q, s = svdq.quantize_act_int8(torch.ones((9, 320), device="cuda:0"), torch.from_numpy(inv).to("cuda:0"))
    assert torch.isnan(s).all() and not q.any()


# narrow rows by 4 to 32 lanes, a wave per row with one to eight chunks, channel counts that vectors of 8 do not divide;
# statistics by one launch and by blocks
@pytest.mark.parametrize("C", [24, 64, 128, 256, 320, 77, 640, 1280, 4096])
@pytest.mark.parametrize("S", [40, 9000])
@pytest.mark.parametrize("act", [svdq.GN_NONE, svdq.GN_SILU, svdq.GN_GELU])
def test_norm_codes(C, S, act):
    """A NaN anywhere in an image's group is in every position of that image, so all of its codes are 0."""
    torch = _torch()
    rng = np.random.default_rng(C)
    x = rng.standard_normal((3, S, C)).astype(np.float32)
    x.view(np.uint32)[0, S // 2, C - 1] = 0xFFC123A5
    x.view(np.uint32)[2, S - 1, 0] = 0x7F8000FF
    q, s = svdq.GroupNorm(C // 7 if C == 77 else 8, C, act=act).quantize(torch.from_numpy(x).to("cuda:0"))
    q, s = q.view(3, S, -1), s.view(3, S)
    assert torch.isnan(s[[0, 2]]).all() and not q[[0, 2]].any()
    assert torch.isfinite(s[1]).all() and q[1].any(1).sum() > 0
    beta = np.zeros(C, np.float32)
    beta.view(np.uint32)[C // 2] = 0x7FC00011
    q, s = svdq.GroupNorm(1, C, beta=beta, act=act).quantize(torch.from_numpy(x[1:2]).to("cuda:0"))
    assert torch.isnan(s).all() and not q.any()
