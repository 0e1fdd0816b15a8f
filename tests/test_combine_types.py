"""moe_combine reads y_packed, gates and dense as fp32: tensors of another type, which the kernel
would read past their end, are refused before the library is called (no GPU is touched)."""
import types

import pytest
import torch

from mixture_experts_layer_57_b200 import moe

STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.fixture
def called(monkeypatch):
    """The library's call replaced by a record of it."""
    calls = []
    fake = types.SimpleNamespace(moe_combine=lambda *a: calls.append(a) or 0,
                                 moe_combine_workspace_bytes=lambda n: 0)
    monkeypatch.setattr(moe, "lib", lambda: fake)
    return calls


def inputs():
    return dict(y_packed=torch.zeros(6, 8), expert_offsets=torch.zeros(3, dtype=torch.int32),
                expert_ids=torch.zeros(4, 1, dtype=torch.int32), slot=torch.zeros(4, 1, dtype=torch.int32),
                gates=torch.zeros(4, 1), dense=torch.zeros(4, 8))


def test_fp32_tensors_are_passed_on(called):
    a = inputs()
    moe.moe_combine(**a, stream=STREAM)
    moe.moe_combine(**dict(a, dense=None), stream=STREAM)
    assert len(called) == 2 and called[0][0] == a["y_packed"].data_ptr()


@pytest.mark.parametrize("name", ["y_packed", "gates", "dense"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float64])
def test_other_types_are_refused(called, name, dtype):
    a = inputs()
    a[name] = a[name].to(dtype)
    with pytest.raises(ValueError, match=name):
        moe.moe_combine(**a, stream=STREAM)
    assert called == []
