"""The library and torch use one HIP runtime in a process, whichever is loaded first (torch brings its own, and device
memory of one means nothing to the other)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MAPPED = """
import sys
print(len({l.split()[-1] for l in open("/proc/self/maps") if "libamdhip64" in l}))
"""


@pytest.mark.parametrize("first", ["svdq.lib()\nimport torch", "import torch\nsvdq.lib()",
                                   "import numpy as np\nsvdq.pack_weights_int8(np.zeros((4, 3), np.uint16))\nimport torch"])
def test_one_runtime_whatever_is_loaded_first(first):
    code = "from bit_diffusion_model_amd import svdq\n" + first + MAPPED
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == ["1"], r.stdout
