"""The block-scaled layer's host pack built for the CPU under AddressSanitizer and UndefinedBehaviorSanitizer (casts of what no
integer holds included) and, separately, ThreadSanitizer, and run with several threads: codes and scales from the formula,
the transpose, and weights with a NaN or an infinity, which are refused without a value being encoded from them.  No GPU:
only pack_fp8.cpp and status.cpp are compiled, with g++."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_diffusion_model_amd", "csrc")

DRIVER = r'''
#include <cmath>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>
#include "svdq.h"
static double value(uint8_t c) {
  const int m = c & 127;
  const double v = m < 8 ? m * 0x1p-9 : (8 + m % 8) * std::ldexp(1.0, m / 8 - 10);
  return c & 128 ? -v : v;
}
int main() {
  std::mt19937 g(3);
  std::normal_distribution<float> d;
  for (int64_t K : {1, 127, 300}) for (int64_t N : {1, 128, 131, 600}) {
    std::vector<uint16_t> W(K * N);
    for (auto& w : W) { float f = d(g); uint32_t u; std::memcpy(&u, &f, 4); w = u >> 16; }
    const int64_t ld = (K + 127) / 128 * 128, kb = ld / 128, ldt = (N + 127) / 128 * 128, nb = ldt / 128;
    std::vector<uint8_t> q(N * ld), t(K * ldt);
    std::vector<float> s(nb * kb), st(kb * nb);
    if (svdq_pack_weights_fp8(K, N, W.data(), q.data(), s.data())) return 1;
    for (int64_t n = 0; n < N; ++n) for (int64_t k = 0; k < ld; ++k) {
      float f = 0.0f;
      if (k < K) { const uint32_t u = (uint32_t)W[k * N + n] << 16; std::memcpy(&f, &u, 4); }
      const double scale = s[n / 128 * kb + k / 128], w = value(q[n * ld + k]) * scale;
      // half a step: 2^-4 of a value, or half of the smallest code
      if (!(std::fabs(w - f) <= std::fmax(std::fabs(f) * 0x1p-4, 0x1p-10 * scale))) return 2;
    }
    if (svdq_transpose_weights_fp8(K, N, q.data(), s.data(), t.data(), st.data())) return 3;
    for (int64_t k = 0; k < K; ++k) for (int64_t n = 0; n < ldt; ++n)
      if (t[k * ldt + n] != (n < N ? q[n * ld + k] : 0)) return 4;
    for (uint16_t bad : {0x7F80, 0xFF80, 0x7FC0, 0x7F81}) for (size_t at : {(size_t)0, W.size() - 1}) {
      const uint16_t was = W[at];
      W[at] = bad;
      if (svdq_pack_weights_fp8(K, N, W.data(), q.data(), s.data()) != SVDQ_ENUMERIC) return 5;
      W[at] = was;
    }
  }
  std::puts("ok");
}
'''


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.parametrize("san", ["address,undefined,float-cast-overflow", "thread"])
def test_pack_under_sanitizer(san, tmp_path):
    src, exe = tmp_path / "driver.cpp", str(tmp_path / "driver")
    src.write_text(DRIVER)
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-pthread", f"-fsanitize={san}",
           "-fno-sanitize-recover=all", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src),
           os.path.join(CSRC, "pack_fp8.cpp"), os.path.join(CSRC, "status.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, env=dict(os.environ, SVDQ_NUM_THREADS="4"), timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, (r.returncode, (r.stdout + r.stderr)[-4000:])
