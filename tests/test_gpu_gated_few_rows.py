"""Few fp32 rows on both sides of the rule that sends them to dot products or to the tiles (rows of an
expert as capacity_hint has them, size of the layer), with a hint that is right, too small and too large."""
import pytest
import torch

from mixture_experts_layer_57_b200 import moe
from tests import gated_ref
from tests.test_gpu_gated_ffn import NAMES, args_of, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[5], [6], [8], [9], [6, 0, 2], [1, 7], [2, 1, 0, 3, 2]], ids=str)
@pytest.mark.parametrize("d,f", [(512, 1024), (513, 1024), (64, 40)])
def test_rule_of_few_rows(cuda_ok, counts, d, f):
    c = make(len(counts), counts, d, f, torch.float32, seed=d + sum(counts), slack=0)
    for hint in (None, 0, 1, 8, 1 << 40):
        y = moe.moe_gated_ffn(args_of(c, "gelu", hint=hint))["y_packed"]
        a = 0
        for e, n in enumerate(counts):
            if n:
                params = {k: c[k][e] for k in NAMES}
                gated_ref.check(f"expert {e}", y[a:a + n],
                                *gated_ref.segment(c["x"][a:a + n], params, "gelu")["y"])
            a += n
