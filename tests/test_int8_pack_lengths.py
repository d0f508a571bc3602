"""The offline helpers of the 8-bit layer refuse arrays that the library would read past the end of (it takes K and N, no
lengths)."""
import numpy as np
import pytest

from bit_diffusion_model_amd import svdq


@pytest.mark.parametrize("n", [0, 1, 99, 101])
def test_pack_needs_one_statistic_per_input_channel(n):
    W = np.zeros((100, 7), np.uint16)
    with pytest.raises(svdq.SvdqError, match="act_absmax"):
        svdq.pack_weights_int8(W, np.ones(n, np.float32))
    with pytest.raises(svdq.SvdqError, match="act_absmax"):
        svdq.pack_weights_int8(W, np.ones((2, n), np.float32))
    for shape in ((100,), (1, 100), (100, 1)):  # a statistic that kept its reduced dimension
        assert svdq.pack_weights_int8(W, np.ones(shape, np.float32))[0].shape == (100,)


def test_pack_needs_a_matrix():
    for W in (np.zeros(100, np.uint16), np.zeros((2, 3, 4), np.uint16)):
        with pytest.raises(svdq.SvdqError, match="W must be"):
            svdq.pack_weights_int8(W)


@pytest.mark.parametrize("shape", [(16, 100), (16, 127), (16, 256), (128,), (2, 16, 128)])
def test_layout_needs_whole_rows_of_codes(shape):
    with pytest.raises(svdq.SvdqError, match="qW"):
        svdq.prepare_weights_int8(100, np.zeros(shape, np.int8))
    assert svdq.prepare_weights_int8(100, np.zeros((16, 128), np.int8)).size == 16 * 128
