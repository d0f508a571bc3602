"""A norm whose gamma and beta are of each image, and there are none: [0][C] is of no image, not one weight for all."""
import numpy as np
import pytest

from bit_diffusion_model_amd import svdq

pytestmark = pytest.mark.gpu


def test_weights_of_no_image():
    import torch

    C = 64
    none = np.zeros((0, C), np.float32)
    for gamma, beta in ((none, none), (none, None), (None, none)):
        ln = svdq.LayerNorm(C, gamma, beta)
        X = torch.ones(0, 5, C, device="cuda:0")
        stats = ln.alloc_stats(X)
        assert ln.forward(X, stats=stats).shape == X.shape
        dX, dg, db = ln.backward(X, X, stats)
        assert dX.shape == X.shape and dg.shape == db.shape == (0, C)
        for shape in ((2, 5, C), (5, C)):  # two images, or one
            Y = torch.ones(shape, device="cuda:0")
            st = ln.alloc_stats(Y)
            for call in (lambda: ln.forward(Y), lambda: ln.quantize(Y), lambda: ln.backward(Y, Y, st)):
                with pytest.raises(svdq.SvdqError, match="0 images"):
                    call()
