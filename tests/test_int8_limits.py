"""The 8-bit layer's documented limits: a launch takes fewer than 2^32 threads.  The quantizer takes any number of rows
(several launches); the product refuses what its grid cannot hold before anything is launched."""
import ctypes

import numpy as np
import pytest

from bit_diffusion_model_amd import svdq
from oracle import int8 as o8


def _err():
    return svdq.lib().svdq_last_error().decode()


# (M, N, what the message names): tiles of 64 x 64 from 2^24 up, blocks of 16 channels from 2^23 up
@pytest.mark.parametrize("M,N,word", [(1 << 30, 64, "2^24"), ((1 << 30) - 63, 1, "2^24"), (1 << 24, 4096, "2^24"),
                                      (1 << 20, 65536, "2^24"), (4, 1 << 27, "2^27"), (1, (1 << 31) - 1, "2^24"),
                                      ((1 << 31) - 1, 1, "2^24"), (40, 1 << 27, "2^27"), (1, (1 << 27) - 15, "2^27")])
def test_refused_before_any_launch(M, N, word):
    """On a host without a GPU a launch would end with status 4; the refusal's is 2."""
    L = svdq.lib()
    lay = svdq._Int8Layer(64, N, 16, 16, 16, 16)
    ref = ctypes.byref(lay)
    assert L.svdq_gemm_w8a8(ref, M, 16, 16, 16, N, 1, 256, 1 << 40, None) == 2 and word in _err()
    assert L.svdq_linear_forward_int8(ref, M, 16, 1, 64, 16, N, 1, 256, 1 << 50, None) == 2 and word in _err()
    assert L.svdq_gemm_w8a8_workspace_bytes(ref, M) == 0 and L.svdq_int8_workspace_bytes(ref, M, 1) == 0
    nrm = svdq._GroupNorm(64, 8, 0, 1e-5, 16, 16)
    args = (ctypes.byref(nrm), ref, 1, M)
    assert L.svdq_norm_linear_forward_int8(*args, 16, 1, 64 * M, 64, 16, N, 1, 256, 1 << 50, None) == 2 and word in _err()
    assert L.svdq_norm_linear_int8_workspace_bytes(*args) == 0


@pytest.mark.parametrize("M,N", [((1 << 30) - 64, 64), (1 << 24, 4032), (100, (1 << 27) - 16)])
def test_largest_sizes_have_a_workspace(M, N):
    lay = svdq._Int8Layer(64, N, 16, 16, 16, 16)
    assert svdq.lib().svdq_int8_workspace_bytes(ctypes.byref(lay), M, 1) >= M * 128 + M * 4


# rows past the 2^32 threads of one launch: four rows to a block of 256 threads, and one
@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [((1 << 26) + 5, 3), ((1 << 24) + 3, 1026)])
def test_quantizer_of_many_rows(M, K):
    import torch

    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda:0")
    edges = [1 << k for k in range(20, 27) if 1 << k < M]
    at = sorted({m for e in [0, M - 1, *edges] for m in range(e - 3, e + 4) if 0 <= m < M})
    rows = torch.tensor(at, device="cuda:0")
    x = np.random.default_rng(K).standard_normal((len(at), K)).astype(np.float32)
    X[rows] = torch.from_numpy(x).to("cuda:0").to(torch.bfloat16)
    qX, sX = svdq.quantize_act_int8(X, out=(torch.full((M, svdq.int8_ld(K)), 5, dtype=torch.int8, device="cuda:0"),
                                            torch.full((M,), 7.0, device="cuda:0")))
    q, s = o8.quantize(X[rows].float().cpu().numpy().astype(np.float64))
    assert np.array_equal(qX[rows].cpu().numpy()[:, :K], q) and np.array_equal(sX[rows].cpu().numpy(), s)
    sX[rows] = float(np.float32(2.0 ** -96) / np.float32(127))
    assert (sX == sX[at[0]]).all(), "a row of zeros without its scale"
    qX[rows] = 0
    part = 1 << 22
    assert not any(qX[m:m + part].any() for m in range(0, M, part)), "a row of zeros without its codes"
    del X, qX, sX
    torch.cuda.empty_cache()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 20])
def test_product_of_many_channels(M):
    """The most channels: weights of 17 GB, of which a few channels are not zero."""
    import torch

    N, K = (1 << 27) - 19, 100
    rng = np.random.default_rng(M)
    at = np.unique(np.concatenate([[0, 1, N - 1, N - 16, N - 17], rng.integers(0, N, 40)]))
    w = rng.integers(-127, 128, (len(at), K)).astype(np.int8)
    qW = torch.zeros((N, 128), dtype=torch.int8, device="cuda:0")
    qW[torch.from_numpy(at).to("cuda:0"), :K] = torch.from_numpy(w).to("cuda:0")
    lin = svdq.Int8Linear(qW, torch.ones(N, device="cuda:0"), K)
    del qW
    x = rng.integers(-127, 128, (M, K)).astype(np.float32)
    x[:, 0] = 127.0  # s = 1: the codes are the values
    Y = lin.forward(torch.from_numpy(x).to("cuda:0"), svdq.F32)
    cols = torch.from_numpy(at).to("cuda:0")
    assert np.array_equal(Y[:, cols].cpu().numpy(), x.astype(np.float64) @ w.astype(np.float64).T)
    Y[:, cols] = 0
    assert not Y.any()
    del lin, Y
    torch.cuda.empty_cache()
