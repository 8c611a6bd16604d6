"""Layer norm launches at every width, whatever ran before it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

# 16-bit widths whose ring fits 48 KB alone, but not with the kernel's own shared memory; ascending, so
# that no wider row has gone before
FRESH = """
import sys
sys.path[:0] = [{here!r}, {root!r}]
import torch
from test_gpu_layer_norm import check, make
for K in (2553, 2601, 2701, 2807):
    check(*make(5, K, torch.{dtype}, torch.float32, seed=K))
print("all right")
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_odd_16_bit_widths_in_a_fresh_process(dtype):
    code = FRESH.format(here=HERE, root=os.path.dirname(HERE), dtype=dtype)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "all right" in r.stdout, r.stderr[-2000:]
