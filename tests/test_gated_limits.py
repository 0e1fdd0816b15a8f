"""Sizes past which the gated FFN's 32-bit row and column arithmetic would wrap are refused on the host
(no GPU is touched)."""
import ctypes

import pytest

from mixture_experts_layer_57_b200 import build as build_mod
from mixture_experts_layer_57_b200 import moe
from tests.test_gated_clip_abi import CUDA, FAKE, UNSUPPORTED, args


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return moe.lib()


@pytest.mark.parametrize("sizes,status", [
    (dict(rows_max=1 << 30), CUDA), (dict(rows_max=(1 << 30) + 1), UNSUPPORTED),
    (dict(rows_max=(1 << 31) - 2), UNSUPPORTED),
    (dict(rows_max=(1 << 31) - 2, dtype=0, out_dtype=0, d_model=1, d_ff=1), UNSUPPORTED),
    (dict(E=1, d_ff=1 << 29), CUDA), (dict(E=1, d_ff=(1 << 29) + 8), UNSUPPORTED),
    (dict(E=1, d_ff=(1 << 31) - 16), UNSUPPORTED), (dict(E=1, d_model=1 << 29), CUDA),
    (dict(E=1, d_model=(1 << 31) - 16), UNSUPPORTED)], ids=str)
def test_size_limits(L, monkeypatch, sizes, status):
    # what passes the checks ends at the injected fault, before anything is enqueued
    monkeypatch.setenv("MOE_FAULT_INJECT", "moe_gated_ffn")
    a = args(**sizes)
    assert L.moe_gated_ffn(ctypes.byref(a), FAKE, FAKE, None, FAKE, 256, None) == status
    monkeypatch.setenv("MOE_FAULT_INJECT", "moe_gated_ffn_backward")
    t = a.dtype
    g = moe.GatedFfnGrads(dx_packed=FAKE, dw_gate=FAKE, dw_up=FAKE, dw_down=FAKE, dx_dtype=t, grad_dtype=t)
    assert L.moe_gated_ffn_backward(ctypes.byref(a), FAKE, FAKE, FAKE, ctypes.byref(g), FAKE, 1 << 62,
                                    None) == status
    n = ctypes.c_size_t()
    assert (L.moe_gated_ffn_backward_workspace_bytes(ctypes.byref(a), ctypes.byref(n)) == UNSUPPORTED) == \
        (status == UNSUPPORTED)
