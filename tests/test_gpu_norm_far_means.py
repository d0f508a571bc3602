"""The layer norm's statistics of rows whose mean lies far from zero, by every number of waves to a row: the bounds of
test_gpu_layer_norm.py, which do not know the mean but for its own rounding (a row's values less a first mean are exact where
they lie within a factor of two of it, and so is the difference of two waves' first means)."""
import numpy as np
import pytest

from bit_diffusion_model_amd import svdq
from oracle import fp8 as o

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


# B S rows of C values: 1, 2, 3, 3, 4, 5, 8, 13, 10 waves of 1 to 4 chunks
@pytest.mark.parametrize("S,C,waves", [(9, 300, 1), (9, 700, 2), (9, 1111, 3), (9, 3001, 3), (9, 2041, 4), (300, 5003, 5),
                                       (9, 8001, 8), (100, 13001, 13), (100, 15001, 10), (3000, 2100, 2)])
@pytest.mark.parametrize("mean,std", [(100.0, 0.05), (-3e4, 1.0), (1.0, 1e-4), (1e4, 1e3)])
def test_statistics(S, C, waves, mean, std):
    import torch

    rng = np.random.default_rng(C)
    x = mean + std * rng.standard_normal((2, S, C))
    x[:, :, C // 3] += 20 * std
    X = torch.from_numpy(x.astype(np.float32)).cuda()
    ln = svdq.LayerNorm(C, eps=1e-30)
    assert ln.plan(2, S)[2] == waves
    stats = ln.alloc_stats(X)
    Y = ln.forward(X, svdq.F32, stats=stats).double().cpu().numpy()
    y, m, r = o.layer_norm(X.double().cpu().numpy(), eps=1e-30)
    gm, gr = (t.double().cpu().numpy().reshape(m.shape) for t in stats)
    off_m, off_r = np.abs(gm - m) / (U * np.abs(m) + 42 * U / r), np.abs(gr - r) / (50 * U * r)
    assert off_m.max() <= 1, f"mean: {off_m.max()} of the bound"
    assert off_r.max() <= 1, f"rstd: {off_r.max()} of the bound"
    tol = r[..., None] * (U * np.abs(m) + 42 * U / r)[..., None] + 58 * U * np.abs(y)
    assert (np.abs(Y - y) <= tol).all()
