"""CPU checks of arithmetic identities the block-scaled quantizer and the layer norm rely on (no GPU involved).

* the scale of a block of 128 values: the fp32 quotient a / 448, formed as a * fp32(1/448) plus one fma correction with the
  exact residual, is the correctly rounded quotient (the scale's definition).  The C check runs every mantissa in twelve
  binades from the smallest to the largest that a block's magnitude can have.
* row r of image b: the launch's reciprocal of S gives floor(r / S) for every row r < 2^31.
"""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_fma_corrected_division_by_448_is_correctly_rounded(tmp_path):
    exe = str(tmp_path / "div448")
    r = subprocess.run(["gcc", "-O2", "-ffp-contract=off", "-o", exe, os.path.join(HERE, "arith", "div448.c"), "-lm"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "0 mismatches", r.stdout[-2000:]


def test_reciprocal_of_the_rows_of_an_image_divides_exactly():
    rng = random.Random(5)
    top = (1 << 31) - 1
    for S in [1, 2, 3, 7, 77, 333, 4608, 65535, 65536, 65537, top - 1, top] + [rng.randrange(1, 1 << rng.randrange(1, 32)) for _ in range(500)]:
        p = 31 + (S - 1).bit_length()
        m = -(-(1 << p) // S)
        rows = [0, top, S - 1, S, S + 1, top // S * S, top // S * S - 1] + [rng.randrange(1 << 31) for _ in range(50)]
        for r in rows:
            if 0 <= r <= top:
                assert r * m < 1 << 64 and (r * m) >> p == r // S, (S, r)
