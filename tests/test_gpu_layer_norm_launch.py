"""Layer norm launches at every width, whatever ran before it and beside it: the shared memory that
a kernel is allowed does not depend on the widths of earlier or concurrent calls."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import moe_expert_layer_count_gb300 as moe

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


def test_two_widths_from_two_threads():
    """Both widths run in one kernel, with 64 and with 48 KB of shared memory."""
    wrong = []
    go = threading.Barrier(2)

    def calls(K):
        try:
            s = torch.cuda.Stream()
            x = torch.randn(1, K, device="cuda").bfloat16()
            w = torch.ones(K, dtype=torch.bfloat16, device="cuda")
            y, mean, rstd = moe.moe_layer_norm(x, w, w)
            torch.cuda.synchronize()
            go.wait(60)
            for _ in range(20000):
                moe.moe_layer_norm(x, w, w, out=y, mean=mean, rstd=rstd, stream=s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            wrong.append(f"K = {K}: {e}")
    threads = [threading.Thread(target=calls, args=(K,)) for K in (8192, 6144)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
