"""Host side of the block-scaled layer and the layer norm (CPU): the pack against the oracle, the transpose, workspace
sizes, and refusals through the C ABI."""
import ctypes

import numpy as np
import pytest

from bit_diffusion_model_amd import svdq
from bit_diffusion_model_amd.workloads import bf16_bits_from_f64, bf16_bits_to_f32
from oracle import fp8 as o

P = ctypes.c_void_p
EINVAL, EUNSUPPORTED, ENUMERIC = 1, 2, 3


def weights(K, N, seed=0):
    rng = np.random.default_rng(seed)
    return bf16_bits_from_f64(rng.standard_normal((K, N)) * np.exp(rng.standard_normal((K, 1))))


@pytest.mark.parametrize("K,N", [(1, 1), (128, 128), (127, 129), (300, 17), (640, 257), (5, 400)])
def test_pack_equals_oracle(K, N):
    W = weights(K, N, K + N)
    q, s = svdq.pack_weights_fp8(W)
    qo, so = o.pack_weights(bf16_bits_to_f32(W).astype(np.float64))
    assert np.array_equal(s, so) and np.array_equal(q, qo)


def test_pack_of_zeros_and_extremes():
    W = np.zeros((256, 130), np.uint16)
    W[3, 129] = 0x7F7F  # the largest bf16
    W[200, 0] = 0x0001  # the smallest
    q, s = svdq.pack_weights_fp8(W)
    qo, so = o.pack_weights(bf16_bits_to_f32(W).astype(np.float64))
    assert np.array_equal(s, so) and np.array_equal(q, qo) and s[0, 0] == 0 and (q[:128, :128] == 0).all()


@pytest.mark.parametrize("K,N", [(1, 1), (128, 256), (127, 129), (300, 17)])
def test_transpose(K, N):
    q, s = svdq.pack_weights_fp8(weights(K, N))
    qt, st = svdq.transpose_weights_fp8(K, q, s)
    assert qt.shape == (K, svdq.int8_ld(N)) and np.array_equal(st, s.T)
    assert np.array_equal(qt[:, :N], q[:, :K].T) and (qt[:, N:] == 0).all()
    q2, s2 = svdq.transpose_weights_fp8(N, qt, st)
    assert np.array_equal(q2, q) and np.array_equal(s2, s)


def test_pack_refusals():
    L = svdq.lib()
    W, q, s = np.zeros((4, 4), np.uint16), np.zeros((4, 128), np.uint8), np.zeros(1, np.float32)
    p = svdq._ptr
    assert L.svdq_pack_weights_fp8(4, 4, None, p(q), p(s)) == EINVAL
    assert L.svdq_pack_weights_fp8(0, 4, p(W), p(q), p(s)) == EINVAL
    assert L.svdq_pack_weights_fp8(4, 0, p(W), p(q), p(s)) == EINVAL
    assert L.svdq_pack_weights_fp8(131073, 4, p(W), p(q), p(s)) == EUNSUPPORTED
    W[1, 2] = 0x7F80
    assert L.svdq_pack_weights_fp8(4, 4, p(W), p(q), p(s)) == ENUMERIC
    assert L.svdq_transpose_weights_fp8(4, 4, None, p(s), p(q), p(s)) == EINVAL
    assert L.svdq_transpose_weights_fp8(4, 131073, p(q), p(s), p(q), p(s)) == EUNSUPPORTED
    with pytest.raises(svdq.SvdqError):
        svdq.pack_weights_fp8(np.zeros(4, np.uint16))
    with pytest.raises(svdq.SvdqError):
        svdq.transpose_weights_fp8(4, q, np.zeros((1, 2), np.float32))


def fake(n=1 << 16):
    """An address that is aligned and never touched: every call below is refused on the host."""
    return n


def layer(K=256, N=256, qW=1 << 16, sW=1 << 16, bias=None):
    return svdq._Fp8Layer(K, N, qW, sW, bias)


@pytest.mark.parametrize("change,want", [
    (dict(layer=None), EINVAL), (dict(layer=layer(K=0)), EINVAL), (dict(layer=layer(N=0)), EINVAL),
    (dict(layer=layer(K=131073)), EUNSUPPORTED), (dict(layer=layer(N=1 << 31)), EUNSUPPORTED),
    (dict(layer=layer(qW=None)), EINVAL), (dict(layer=layer(sW=None)), EINVAL), (dict(layer=layer(qW=(1 << 16) + 8)), EINVAL),
    (dict(layer=layer(bias=(1 << 16) + 4)), EINVAL), (dict(M=-1), EINVAL), (dict(M=1 << 31), EUNSUPPORTED),
    (dict(X=None), EINVAL), (dict(X=(1 << 16) + 1), EINVAL), (dict(xdtype=2), EUNSUPPORTED), (dict(ldx=255), EINVAL),
    (dict(ldx=1 << 31), EUNSUPPORTED), (dict(Y=None), EINVAL), (dict(ydtype=3), EUNSUPPORTED), (dict(ldy=255), EINVAL),
    (dict(ldy=1 << 31), EUNSUPPORTED), (dict(ws=None), EINVAL), (dict(ws=(1 << 16) + 128), EINVAL), (dict(ws_bytes=64), EINVAL),
    (dict(layer=layer(N=(1 << 27) - 15)), EUNSUPPORTED), (dict(M=1 << 30, layer=layer(N=1 << 20)), EUNSUPPORTED),
])
def test_layer_refusals(change, want):
    a = dict(layer=layer(), M=64, X=fake(), xdtype=1, ldx=256, Y=fake(), ldy=1 << 28, ydtype=0, ws=fake(), ws_bytes=1 << 40) | change
    lay = ctypes.byref(a["layer"]) if a["layer"] is not None else None
    r = svdq.lib().svdq_linear_forward_fp8(lay, a["M"], a["X"], a["xdtype"], a["ldx"], a["Y"], a["ldy"], a["ydtype"], a["ws"],
                                           a["ws_bytes"], None)
    assert r == want, svdq.lib().svdq_last_error()
    assert svdq.lib().svdq_last_error() != b""


def test_product_and_quantizer_refusals():
    L, lay = svdq.lib(), layer()
    r = ctypes.byref(lay)
    assert L.svdq_gemm_fp8(r, 64, None, fake(), fake(), 256, 0, None, 0, None) == EINVAL
    assert L.svdq_gemm_fp8(r, 64, fake(), fake() + 4, fake(), 256, 0, None, 0, None) == EINVAL
    assert L.svdq_gemm_fp8(r, 64, fake() + 8, fake(), fake(), 256, 0, None, 0, None) == EINVAL
    assert L.svdq_gemm_fp8(r, 0, None, None, None, 0, 0, None, 0, None) == 0
    assert L.svdq_quantize_act_fp8(64, 0, fake(), 0, 256, fake(), fake(), None) == EINVAL
    assert L.svdq_quantize_act_fp8(64, 256, fake(), 2, 256, fake(), fake(), None) == EUNSUPPORTED
    assert L.svdq_quantize_act_fp8(64, 256, fake(), 1, 255, fake(), fake(), None) == EINVAL
    assert L.svdq_quantize_act_fp8(64, 256, fake(), 1, 256, fake() + 8, fake(), None) == EINVAL
    assert L.svdq_quantize_act_fp8(0, 256, None, 1, 256, None, None, None) == 0
    p = (ctypes.c_int32 * 4)()
    assert L.svdq_debug_fp8_plan(r, 0, 0, p) == EINVAL
    assert L.svdq_fp8_workspace_bytes(r, 0) == 0 and L.svdq_fp8_workspace_bytes(None, 64) == 0
    assert L.svdq_fp8_workspace_bytes(r, 64) >= 64 * 256 + 2 * 64 * 4


def norm(C=256, eps=1e-5, one_plus=0, gamma=None, beta=None, stride=0):
    return svdq._LayerNorm(C, eps, one_plus, gamma, beta, stride)


NORM = [
    (dict(norm=None), EINVAL), (dict(norm=norm(C=0)), EINVAL), (dict(norm=norm(C=16385)), EUNSUPPORTED),
    (dict(norm=norm(eps=0.0)), EINVAL), (dict(norm=norm(eps=float("nan"))), EINVAL), (dict(norm=norm(one_plus=2)), EINVAL),
    (dict(norm=norm(gamma=(1 << 16) + 2)), EINVAL), (dict(norm=norm(stride=255)), EINVAL),
    (dict(norm=norm(stride=1 << 46)), EUNSUPPORTED), (dict(B=-1), EINVAL), (dict(B=65536), EUNSUPPORTED),
    (dict(S=1 << 31), EUNSUPPORTED), (dict(X=None), EINVAL), (dict(xdtype=2), EUNSUPPORTED), (dict(ldx=255), EINVAL),
    (dict(bsx=100), EINVAL), (dict(bsx=-1), EINVAL), (dict(bsx=1 << 46), EUNSUPPORTED), (dict(mean=(1 << 16) + 1), EINVAL),
]


@pytest.mark.parametrize("change,want", NORM + [(dict(Y=None), EINVAL), (dict(ydtype=2), EUNSUPPORTED), (dict(ldy=255), EINVAL),
                                                (dict(bsy=0), EINVAL), (dict(bsy=1 << 46), EUNSUPPORTED)])
def test_norm_refusals(change, want):
    a = dict(norm=norm(), B=2, S=10, X=fake(), xdtype=1, bsx=2560, ldx=256, Y=fake(), ydtype=1, bsy=2560, ldy=256, mean=None) | change
    n = ctypes.byref(a["norm"]) if a["norm"] is not None else None
    r = svdq.lib().svdq_layer_norm(n, a["B"], a["S"], a["X"], a["xdtype"], a["bsx"], a["ldx"], a["Y"], a["ydtype"], a["bsy"],
                                   a["ldy"], a["mean"], None, None)
    assert r == want, svdq.lib().svdq_last_error()


@pytest.mark.parametrize("change,want", NORM + [
    (dict(dY=None), EINVAL), (dict(dY=(1 << 16) + 1), EINVAL), (dict(dydtype=2), EUNSUPPORTED), (dict(lddy=255), EINVAL),
    (dict(bsdy=3), EINVAL), (dict(mean=None), EINVAL), (dict(rstd=None), EINVAL), (dict(dX=None), EINVAL),
    (dict(lddx=255), EINVAL), (dict(bsdx=0), EINVAL), (dict(lddx=1 << 31), EUNSUPPORTED), (dict(dgamma=(1 << 16) + 2), EINVAL),
    (dict(ws=None), EINVAL), (dict(ws=(1 << 16) + 64), EINVAL), (dict(ws_bytes=8), EINVAL)])
def test_gradient_refusals(change, want):
    a = dict(norm=norm(), B=2, S=100000, dY=fake(), dydtype=0, bsdy=25600000, lddy=256, X=fake(), xdtype=1, bsx=25600000, ldx=256,
             mean=fake(), rstd=fake(), dX=fake(), bsdx=25600000, lddx=256, dgamma=fake(), dbeta=fake(), ws=fake(),
             ws_bytes=1 << 40) | change
    n = ctypes.byref(a["norm"]) if a["norm"] is not None else None
    r = svdq.lib().svdq_layer_norm_backward(n, a["B"], a["S"], a["dY"], a["dydtype"], a["bsdy"], a["lddy"], a["X"], a["xdtype"],
                                            a["bsx"], a["ldx"], a["mean"], a["rstd"], a["dX"], a["bsdx"], a["lddx"], a["dgamma"],
                                            a["dbeta"], a["ws"], a["ws_bytes"], None)
    assert r == want, svdq.lib().svdq_last_error()


def test_norm_and_layer_refusals():
    L, n, lay = svdq.lib(), norm(), layer(K=255)

    def call(lay, X=fake(), ws=fake()):
        return L.svdq_norm_linear_forward_fp8(ctypes.byref(n), ctypes.byref(lay), 1, 8, X, 1, 0, 256, fake(), 256, 0, None,
                                              None, ws, 1 << 40, None)

    assert call(lay) == EINVAL and b"must equal" in L.svdq_last_error()
    assert call(layer(), X=None) == EINVAL and call(layer(), ws=None) == EINVAL
    assert L.svdq_norm_linear_fp8_workspace_bytes(ctypes.byref(n), ctypes.byref(lay), 1, 8) == 0
    assert L.svdq_norm_linear_fp8_workspace_bytes(ctypes.byref(n), ctypes.byref(layer()), 1, 8) >= 8 * 256 + 2 * 8 * 4
    assert L.svdq_layer_norm(ctypes.byref(n), 0, 5, None, 0, 0, 0, None, 0, 0, 0, None, None, None) == 0
    assert L.svdq_layer_norm_backward_workspace_bytes(ctypes.byref(n), 0, 5) == 0
