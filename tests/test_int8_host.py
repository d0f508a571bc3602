"""Host-side tests of the 8-bit layer and the group norm (no GPU): the library's pack against oracle/int8.py, the
kernel layout of the weights, and the checks of arguments of every entry point."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from bit_diffusion_model_amd import svdq
from bit_diffusion_model_amd.workloads import bf16_bits_from_f64, bf16_bits_to_f32
from oracle import int8 as o8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_diffusion_model_amd", "csrc")


def _err():
    return svdq.lib().svdq_last_error().decode()


@pytest.mark.parametrize("K,N", [(1, 1), (7, 3), (128, 64), (130, 65), (1000, 77)])
@pytest.mark.parametrize("smooth", [False, True])
def test_pack_matches_oracle(K, N, smooth):
    rng = np.random.default_rng(K + N)
    W = rng.standard_normal((K, N)) * 10.0 ** rng.uniform(-3, 3, (1, N))
    W[:, 0] = 0.0
    bits = bf16_bits_from_f64(W)
    a = (10.0 ** rng.uniform(-3, 2, K)).astype(np.float32) if smooth else None
    s, inv, qW, sW = svdq.pack_weights_int8(bits, a, 0.5)
    so, invo, qo, swo = o8.pack_weights(bf16_bits_to_f32(bits), a, 0.5)
    # sqrt(a) / sqrt(w) in fp64 by two C libraries: the same fp32 unless it lies on a rounding boundary
    assert np.abs(s / so - 1).max() <= 2.0 ** -23
    np.testing.assert_array_equal(inv, (np.float32(1) / s))
    same = s == so  # the codes are decided by the library's own s
    What = s.astype(np.float64)[:, None] * bf16_bits_to_f32(bits)
    np.testing.assert_array_equal(sW, (np.abs(What).max(0) / 127.0).astype(np.float32))
    d = np.where(sW == 0, 1.0, sW.astype(np.float64))
    np.testing.assert_array_equal(qW[:, :K], (np.rint(What / d) * (sW != 0)).T)
    assert (qW[:, K:] == 0).all() and (qW[0] == 0).all() and sW[0] == 0
    if same.all():
        np.testing.assert_array_equal(qW, qo)
        np.testing.assert_array_equal(sW, swo)


def test_pack_refusals():
    W = np.zeros((4, 3), np.uint16)
    with pytest.raises(svdq.SvdqError):
        svdq.pack_weights_int8(W, np.ones(4, np.float32), 1.5)
    bad = W.copy()
    bad[2, 1] = 0x7FC0
    with pytest.raises(svdq.SvdqError, match="finite"):
        svdq.pack_weights_int8(bad)
    with pytest.raises(svdq.SvdqError, match="finite"):
        svdq.pack_weights_int8(W, np.array([1, np.inf, 1, 1], np.float32))
    L = svdq.lib()
    assert L.svdq_pack_weights_int8(4, 3, None, None, 0.5, 16, 16, 16, 16) == 1
    assert L.svdq_pack_weights_int8(0, 3, 16, None, 0.5, 16, 16, 16, 16) == 1
    assert L.svdq_pack_weights_int8(1 << 18, 3, 16, None, 0.5, 16, 16, 16, 16) == 2
    assert L.svdq_prepare_weights_int8(4, 3, None, 16) == 1 and L.svdq_prepare_weights_int8(4, 0, 16, 16) == 1
    assert L.svdq_prepare_weights_int8(1 << 18, 3, 16, 16) == 2


@pytest.mark.parametrize("K,N", [(1, 1), (100, 16), (128, 17), (300, 40)])
def test_kernel_layout(K, N):
    """Code (n, k) at (n / 16) 16 ld + (k / 64) 1024 + ((k / 16) % 4) 256 + (n % 16) 16 + k % 16, padding zero."""
    ld = svdq.int8_ld(K)
    assert ld == o8.ld(K) == svdq.lib().svdq_int8_ld(K)
    q = np.zeros((N, ld), np.int8)
    q[:, :K] = np.random.default_rng(N).integers(-127, 128, (N, K))
    out = svdq.prepare_weights_int8(K, q)
    assert out.size == (N + 15) // 16 * 16 * ld
    n, k = np.meshgrid(np.arange(N), np.arange(ld), indexing="ij")
    at = (n // 16) * 16 * ld + (k // 64) * 1024 + ((k // 16) % 4) * 256 + (n % 16) * 16 + k % 16
    np.testing.assert_array_equal(out[at], q)
    rest = np.ones(out.size, bool)
    rest[at] = False
    assert (out[rest] == 0).all()


def test_layer_entry_points_validate_on_host():
    L = svdq.lib()
    lay = svdq._Int8Layer(256, 64, 16, 16, 16, 16)  # fake aligned non-NULL pointers
    ref = ctypes.byref(lay)
    # no rows: a no-op that never touches the device
    assert L.svdq_quantize_act_int8(0, 256, None, 1, 256, None, None, None, None) == 0
    assert L.svdq_gemm_w8a8(ref, 0, None, None, None, 64, 0, None, 0, None) == 0
    assert L.svdq_linear_forward_int8(ref, 0, None, 1, 256, None, 64, 0, None, 0, None) == 0
    # NULL, sizes, types, strides, alignment, limits
    assert L.svdq_quantize_act_int8(4, 0, 16, 1, 256, None, 16, 16, None) == 1
    assert L.svdq_quantize_act_int8(4, 1 << 18, 16, 1, 1 << 18, None, 16, 16, None) == 2
    assert L.svdq_quantize_act_int8(-1, 256, 16, 1, 256, None, 16, 16, None) == 1
    assert L.svdq_quantize_act_int8(4, 256, None, 1, 256, None, 16, 16, None) == 1
    assert L.svdq_quantize_act_int8(4, 256, 16, 2, 256, None, 16, 16, None) == 2 and "dtype" in _err()
    assert L.svdq_quantize_act_int8(4, 256, 16, 1, 255, None, 16, 16, None) == 1 and "ldx" in _err()
    assert L.svdq_quantize_act_int8(4, 256, 17, 1, 256, None, 16, 16, None) == 1 and "aligned" in _err()
    assert L.svdq_quantize_act_int8(4, 256, 18, 0, 256, None, 16, 16, None) == 1 and "aligned" in _err()
    assert L.svdq_quantize_act_int8(4, 256, 16, 1, 256, 8, 16, 16, None) == 1 and "inv_s" in _err()
    assert L.svdq_quantize_act_int8(4, 256, 16, 1, 256, None, 8, 16, None) == 1 and "qX" in _err()
    assert L.svdq_quantize_act_int8(4, 256, 16, 1, 1 << 31, None, 16, 16, None) == 2 and "ldx" in _err()
    assert L.svdq_gemm_w8a8(None, 4, 16, 16, 16, 64, 0, None, 0, None) == 1
    assert L.svdq_gemm_w8a8(ref, 4, 16, None, 16, 64, 0, None, 0, None) == 1
    assert L.svdq_gemm_w8a8(ref, 4, 16, 16, 16, 63, 0, None, 0, None) == 1 and "ldy" in _err()
    assert L.svdq_gemm_w8a8(ref, 4, 16, 16, 16, 64, 3, None, 0, None) == 2 and "dtype" in _err()
    assert L.svdq_gemm_w8a8(ref, 4, 16, 16, 18, 64, 0, None, 0, None) == 1 and "Y" in _err()
    huge = svdq._Int8Layer(256, 1 << 30, 16, 16, 16, 16)
    assert L.svdq_gemm_w8a8(ctypes.byref(huge), 1 << 30, 16, 16, 16, 1 << 30, 0, None, 0, None) == 2 and "2^43" in _err()
    for bad, st in ((svdq._Int8Layer(0, 64, 16, 16, 16, 16), 1), (svdq._Int8Layer(256, 0, 16, 16, 16, 16), 1),
                    (svdq._Int8Layer(1 << 18, 64, 16, 16, 16, 16), 2), (svdq._Int8Layer(256, 64, 16, None, 16, 16), 1),
                    (svdq._Int8Layer(256, 64, 16, 16, None, 16), 1), (svdq._Int8Layer(256, 64, 8, 16, 16, 16), 1),
                    (svdq._Int8Layer(256, 64, 16, 16, 16, 8), 1)):
        assert L.svdq_gemm_w8a8(ctypes.byref(bad), 4, 16, 16, 16, 64, 0, None, 0, None) == st
        assert L.svdq_linear_forward_int8(ctypes.byref(bad), 4, 16, 1, 256, 16, 64, 0, 256, 1 << 30, None) == st
    # workspaces: none for few tokens, the codes and scales beyond, and refused where too small
    assert L.svdq_int8_workspace_bytes(ref, 1, 1) == 0
    need = L.svdq_int8_workspace_bytes(ref, 100, 1)
    assert need >= 100 * 256 + 400
    assert L.svdq_linear_forward_int8(ref, 100, 16, 1, 256, 16, 64, 0, 256, need - 1, None) == 1 and "workspace" in _err()
    assert L.svdq_linear_forward_int8(ref, 100, 16, 1, 256, 16, 64, 0, 128, need, None) == 1 and "workspace" in _err()
    assert L.svdq_int8_workspace_bytes(None, 4, 1) == 0 and L.svdq_int8_workspace_bytes(ref, 4, 7) == 0


def test_norm_entry_points_validate_on_host():
    L = svdq.lib()
    nrm = svdq._GroupNorm(64, 8, 1, 1e-5, 16, 16)
    ref = ctypes.byref(nrm)
    ws = (256, 1 << 30)
    ok = lambda n=ref, B=2, S=8000, X=16, xd=1, bsx=512000, ldx=64, Y=16, yd=1, bsy=512000, ldy=64, w=ws: L.svdq_group_norm(  # noqa: E731
        n, B, S, X, xd, bsx, ldx, Y, yd, bsy, ldy, *w, None)
    assert ok(B=0, X=None, Y=None) == 0 and ok(S=0, X=None, Y=None) == 0
    assert ok(n=None) == 1 and ok(B=-1) == 1 and ok(S=-1) == 1
    assert ok(X=None) == 1 and ok(Y=None) == 1 and ok(X=17) == 1 and ok(Y=18, yd=0) == 1
    assert ok(xd=2) == 2 and ok(yd=2) == 2 and ok(xd=7) == 2
    assert ok(ldx=63) == 1 and ok(ldy=63) == 1 and ok(bsx=511999) == 1 and "bsx" in _err()
    assert ok(bsy=511000) == 1 and "bsy" in _err()
    assert ok(B=70000, S=1) == 2 and ok(ldx=1 << 31, bsx=1 << 40) == 2
    assert ok(w=(256, 8)) == 1 and "workspace" in _err() and ok(w=(128, 1 << 30)) == 1 and ok(w=(None, 0)) == 1
    # a group that fits one block needs no workspace, its codes' statistics do
    assert L.svdq_group_norm_workspace_bytes(ref, 2, 10) == 0 < L.svdq_group_norm_quantize_workspace_bytes(ref, 2, 10)
    for bad, st in (((0, 8, 1, 1e-5, 16, 16), 1), ((64, 0, 1, 1e-5, 16, 16), 1), ((64, 7, 1, 1e-5, 16, 16), 1),
                    ((8192, 8, 1, 1e-5, 16, 16), 2), ((4096, 2048, 1, 1e-5, 16, 16), 2), ((64, 8, 3, 1e-5, 16, 16), 2),
                    ((64, 8, 1, 0.0, 16, 16), 1), ((64, 8, 1, float("nan"), 16, 16), 1), ((64, 8, 1, 1e-5, 8, 16), 1),
                    ((64, 8, 1, 1e-5, 16, 8), 1)):
        assert ok(n=ctypes.byref(svdq._GroupNorm(*bad)), ldx=8192, bsx=8192 * 8000, ldy=8192, bsy=8192 * 8000) == st, bad
        assert L.svdq_group_norm_workspace_bytes(ctypes.byref(svdq._GroupNorm(*bad)), 2, 10) == 0
    q = lambda inv=16, qX=16, sX=16, w=ws: L.svdq_group_norm_quantize_int8(ref, 2, 10, 16, 1, 640, 64, inv, qX, sX, *w, None)  # noqa: E731
    assert q(inv=8) == 1 and q(qX=None) == 1 and q(qX=8) == 1 and q(sX=None) == 1 and q(w=(256, 8)) == 1
    lay = svdq._Int8Layer(64, 32, 16, 16, 16, 16)
    other = svdq._Int8Layer(65, 32, 16, 16, 16, 16)
    f = lambda l, w=ws, ldy=32: L.svdq_norm_linear_forward_int8(ref, ctypes.byref(l), 2, 10, 16, 1, 640, 64, 16, ldy, 1, *w, None)  # noqa: E731
    assert f(other) == 1 and "K" in _err() and f(lay, ldy=31) == 1 and f(lay, w=(256, 64)) == 1
    assert L.svdq_norm_linear_int8_workspace_bytes(ref, ctypes.byref(other), 2, 10) == 0
    assert L.svdq_norm_linear_int8_workspace_bytes(ref, ctypes.byref(lay), 2, 10) >= 20 * 128 + 80


def test_launch_failure_reports_hip_error():
    import torch

    if torch.cuda.is_available():
        pytest.skip("needs a host without a visible GPU")
    L = svdq.lib()
    lay = svdq._Int8Layer(256, 64, 16, 16, 16, 16)
    assert L.svdq_quantize_act_int8(4, 256, 16, 1, 256, None, 16, 16, None) == 4 and "launch" in _err()
    assert L.svdq_gemm_w8a8(ctypes.byref(lay), 400, 16, 16, 16, 64, 0, 256, 1 << 30, None) == 4 and "launch" in _err()
    assert L.svdq_linear_forward_int8(ctypes.byref(lay), 2, 16, 1, 256, 16, 64, 0, None, 0, None) == 4
    nrm = svdq._GroupNorm(64, 8, 1, 1e-5, 16, 16)
    assert L.svdq_group_norm(ctypes.byref(nrm), 2, 10, 16, 1, 640, 64, 16, 1, 640, 64, 256, 1 << 30, None) == 4


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.parametrize("san", ["address,undefined", "thread"])
def test_host_pack_under_sanitizer(san, tmp_path):
    """pack_int8.cpp driven with several threads under the sanitizers, its output checked against a plain loop."""
    src = tmp_path / "driver.cpp"
    src.write_text(r'''
#include <cmath>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>
#include "svdq.h"
int main() {
  std::mt19937 g(3);
  std::normal_distribution<float> d;
  for (int64_t K : {1, 65, 300}) for (int64_t N : {1, 70, 130}) {
    std::vector<uint16_t> W(K * N);
    for (auto& w : W) { float f = d(g); uint32_t u; std::memcpy(&u, &f, 4); w = u >> 16; }
    std::vector<float> a(K, 2.0f), s(K), inv(K), sw(N);
    const int64_t ld = svdq_int8_ld(K);
    std::vector<int8_t> q(N * ld), o(svdq_int8_weight_bytes(K, N));
    if (svdq_pack_weights_int8(K, N, W.data(), a.data(), 0.5f, s.data(), inv.data(), q.data(), sw.data())) return 1;
    if (svdq_prepare_weights_int8(K, N, q.data(), o.data())) return 2;
    for (int64_t n = 0; n < N; ++n) for (int64_t k = 0; k < K; ++k) {
      uint32_t u = (uint32_t)W[k * N + n] << 16; float f; std::memcpy(&f, &u, 4);
      if (q[n * ld + k] != (int8_t)std::nearbyint((double)s[k] * f / (double)sw[n])) return 3;
      if (o[n / 16 * 16 * ld + k / 64 * 1024 + k / 16 % 4 * 256 + n % 16 * 16 + k % 16] != q[n * ld + k]) return 4;
    }
    W[K * N - 1] = 0x7F80;
    if (svdq_pack_weights_int8(K, N, W.data(), nullptr, 0.5f, s.data(), inv.data(), q.data(), sw.data()) != SVDQ_ENUMERIC) return 5;
  }
  std::puts("ok");
}
''')
    exe = str(tmp_path / "driver")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-pthread", f"-fsanitize={san}",
           "-fno-sanitize-recover=all", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src),
           os.path.join(CSRC, "pack_int8.cpp"), os.path.join(CSRC, "status.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, env=dict(os.environ, SVDQ_NUM_THREADS="4"), timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, (r.stdout + r.stderr)[-4000:]
