"""The gated FFN where the device holds no thread-block clusters (a context of few SMs): the host is
told so, in a process of its own as the answer is kept, and every product has to run on single CTAs."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import torch
from mixture_experts_layer_57_b200 import moe
from tests import gated_ref
from tests.test_gpu_gated_ffn import NAMES, args_of, make
# one row and few rows of a wide block (split sums), many rows (pairs), short sums, fp32
for counts, d, f, dtype in (([1], 1024, 2056, torch.bfloat16), ([100, 0, 30], 512, 776, torch.bfloat16),
                            ([300, 129], 256, 520, torch.bfloat16), ([40], 64, 72, torch.bfloat16),
                            ([20], 301, 700, torch.float32)):
    c = make(len(counts), counts, d, f, dtype, seed=d)
    r = moe.moe_gated_ffn(args_of(c), train=True)
    assert moe.moe_get_device_error(r["ws"]) == 0
    a = 0
    for e, n in enumerate(counts):
        if n:
            params = {k: c[k][e] for k in NAMES}
            gated_ref.check("y", r["y_packed"][a:a + n], *gated_ref.segment(c["x"][a:a + n], params, "silu")["y"])
        a += n
print("all right")
"""


def test_no_clusters(cuda_ok):
    env = dict(os.environ, MOE_FAULT_INJECT="clusters", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, cwd=ROOT, env=env,
                       timeout=300)
    assert r.returncode == 0 and "all right" in r.stdout, r.stdout + r.stderr
