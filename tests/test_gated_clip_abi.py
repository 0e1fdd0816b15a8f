"""Refusals of the gated FFN and gradient-clipping entry points, on the host (no GPU is touched:
validation fails before any CUDA call)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_57_b200 import build as build_mod
from mixture_experts_layer_57_b200 import moe

FAKE = 0x10000  # aligned, never dereferenced
OK, INVALID, UNSUPPORTED, SMALL, CUDA, MISALIGNED = 0, 1, 2, 3, 4, 6


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return moe.lib()


def args(**kw):
    a = dict(x_packed=FAKE, expert_offsets=FAKE, E=4, rows_max=16, d_model=64, d_ff=128, dtype=1,
             out_dtype=1, act=0, w_gate=FAKE, w_up=FAKE, w_down=FAKE, capacity_hint=16)
    a.update(kw)
    return moe.GatedFfnArgs(**a)


def test_gated_forward_refusals(L, monkeypatch):
    def call(h=FAKE, y=FAKE, saved=None, ws=FAKE, wsb=256, **kw):
        return L.moe_gated_ffn(ctypes.byref(args(**kw)), h, y, saved, ws, wsb, None)
    assert L.moe_gated_ffn(None, FAKE, FAKE, None, FAKE, 256, None) == INVALID
    for name in ("x_packed", "expert_offsets", "w_gate", "w_up", "w_down"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: FAKE + 8}) == MISALIGNED
    for name in ("b_gate", "b_up", "b_down"):
        assert call(**{name: FAKE + 2}) == MISALIGNED
    assert call(E=0) == INVALID and call(rows_max=-1) == INVALID and call(d_ff=0) == INVALID
    assert call(dtype=2) == INVALID and call(out_dtype=5) == INVALID
    assert call(act=2) == INVALID and call(act=-1) == INVALID
    assert call(capacity_hint=-1) == INVALID
    assert call(E=1025) == UNSUPPORTED and call(rows_max=1 << 31) == UNSUPPORTED
    assert call(d_model=60) == UNSUPPORTED and call(d_ff=100) == UNSUPPORTED
    assert call(dtype=0, out_dtype=1) == UNSUPPORTED        # fp32 layers write fp32
    assert call(dtype=0, out_dtype=0, d_model=20000) == UNSUPPORTED
    assert call(h=None) == INVALID and call(y=None) == INVALID and call(ws=None) == INVALID
    assert call(h=FAKE + 4) == MISALIGNED and call(saved=FAKE + 2) == MISALIGNED
    assert call(ws=FAKE + 16) == MISALIGNED and call(wsb=255) == SMALL
    monkeypatch.setenv("MOE_FAULT_INJECT", "moe_gated_ffn")
    assert call() == CUDA and call(act=9) == INVALID
    monkeypatch.setenv("MOE_FAULT_INJECT", "moe_expert_ffn")
    assert call(rows_max=0) == OK                           # nothing is enqueued


def test_gated_backward_refusals(L, monkeypatch):
    need = moe.moe_gated_ffn_backward_workspace_bytes(args())
    assert need >= 256 + 2 * 16 * 128 * 2                   # dg and du

    def call(dy=FAKE, h=FAKE, saved=FAKE, ws=FAKE, wsb=need, a=None, **kw):
        g = dict(dx_packed=FAKE, dw_gate=FAKE, dw_up=FAKE, dw_down=FAKE, dx_dtype=1, grad_dtype=1)
        g.update(kw)
        return L.moe_gated_ffn_backward(ctypes.byref(args(**(a or {}))), dy, h, saved,
                                        ctypes.byref(moe.GatedFfnGrads(**g)), ws, wsb, None)
    assert L.moe_gated_ffn_backward(ctypes.byref(args()), FAKE, FAKE, FAKE, None, FAKE, need,
                                    None) == INVALID
    assert call(dy=None) == INVALID and call(h=None) == INVALID and call(saved=None) == INVALID
    for name in ("dx_packed", "dw_gate", "dw_up", "dw_down"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: FAKE + 4}) == MISALIGNED
    for name in ("db_gate", "db_up", "db_down"):
        assert call(**{name: FAKE + 4}) == MISALIGNED
    assert call(dy=FAKE + 4) == MISALIGNED
    assert call(dx_dtype=3) == INVALID and call(grad_dtype=-1) == INVALID
    f32 = dict(dtype=0, out_dtype=0)
    big = 1 << 30
    assert call(a=f32, wsb=big, dx_dtype=1, grad_dtype=0) == UNSUPPORTED
    assert call(a=f32, wsb=big, dx_dtype=0, grad_dtype=1) == UNSUPPORTED
    assert call(a=dict(act=7)) == INVALID
    assert call(wsb=need - 1) == SMALL
    monkeypatch.setenv("MOE_FAULT_INJECT", "moe_gated_ffn_backward")
    assert call() == CUDA
    n = ctypes.c_size_t()
    assert L.moe_gated_ffn_backward_workspace_bytes(None, ctypes.byref(n)) == INVALID
    assert L.moe_gated_ffn_backward_workspace_bytes(ctypes.byref(args(d_ff=4)), ctypes.byref(n)) == UNSUPPORTED


def grads(*rows):
    return (moe.GradTensor * len(rows))(*rows), len(rows)


def test_norm_and_clip_refusals(L, monkeypatch):
    need = moe.moe_grad_norm_workspace_bytes()
    F32, BF16 = 0, 1
    one = (FAKE, FAKE, 100, F32, F32)

    def norm(rows=(one,), out=FAKE * 8, ws=FAKE, wsb=need):
        t, n = grads(*rows)
        return L.moe_grad_norm(t, n, out, ws, wsb, None)

    def clip(rows=(one,), nrm=FAKE * 8, m=1.0):
        t, n = grads(*rows)
        return L.moe_clip_grads(t, n, nrm, m, None)
    assert L.moe_grad_norm(None, 1, FAKE, FAKE, need, None) == INVALID
    assert L.moe_grad_norm(None, -1, FAKE, FAKE, need, None) == INVALID
    assert L.moe_clip_grads(None, 1, FAKE, 1.0, None) == INVALID
    assert norm(out=None) == INVALID and norm(ws=None) == INVALID
    assert norm(out=FAKE + 2) == MISALIGNED and norm(ws=FAKE + 16) == MISALIGNED
    assert norm(wsb=need - 1) == SMALL
    for call in (norm, clip):
        assert call([(None, FAKE, 4, F32, F32)]) == INVALID
        assert call([(FAKE, FAKE, -1, F32, F32)]) == INVALID
        assert call([(FAKE, FAKE, 4, 2, F32)]) == INVALID
        assert call([(FAKE + 2, FAKE, 4, F32, F32)]) == MISALIGNED
        assert call([(FAKE + 1, FAKE, 4, BF16, F32)]) == MISALIGNED
        assert call([(FAKE, FAKE, 1 << 43, F32, F32)]) == UNSUPPORTED
    assert clip([(FAKE, None, 4, F32, F32)]) == INVALID
    assert clip([(FAKE, FAKE * 2, 4, F32, 7)]) == INVALID
    assert clip([(FAKE, FAKE * 2 + 2, 4, F32, F32)]) == MISALIGNED
    assert clip(nrm=None) == INVALID and clip(nrm=FAKE + 1) == MISALIGNED
    for m in (-1.0, float("inf"), float("nan")):
        assert clip(m=m) == INVALID
    # outputs that overlap: a tensor listed twice, halves of one buffer, another's gradient, a
    # narrower type in place, the norm itself
    assert clip([one, one]) == INVALID
    assert clip([(FAKE, FAKE * 2, 100, F32, F32), (FAKE * 3, FAKE * 2 + 396, 10, F32, F32)]) == INVALID
    assert clip([(FAKE, FAKE * 2, 100, F32, F32), (FAKE * 2 + 4, FAKE * 4, 10, F32, F32)]) == INVALID
    assert clip([(FAKE, FAKE, 100, F32, BF16)]) == INVALID
    assert clip(nrm=FAKE + 396) == INVALID
    monkeypatch.setenv("MOE_FAULT_INJECT", "moe_grad_norm")
    assert norm() == CUDA
    monkeypatch.setenv("MOE_FAULT_INJECT", "moe_clip_grads")
    assert clip() == CUDA
    # neighbours that only touch, and a gradient read twice into two places, are fine
    assert clip([(FAKE, FAKE, 100, F32, F32), (FAKE + 400, FAKE + 400, 100, F32, F32)]) == CUDA
    assert clip([(FAKE, FAKE * 2, 100, F32, F32), (FAKE, FAKE * 3, 100, F32, F32)]) == CUDA


def test_binding_refusals():
    bf = dict(dtype=torch.bfloat16)
    x, off = torch.zeros(6, 16, **bf), torch.zeros(3, dtype=torch.int32)
    wg, wd = torch.zeros(2, 24, 16, **bf), torch.zeros(2, 16, 24, **bf)
    moe.gated_ffn_args(x, off, wg, wg, wd)
    for bad in (dict(act="relu"), dict(rows_max=7), dict(out_dtype=torch.float16),
                dict(b_gate=torch.zeros(2, 16, **bf)), dict(b_down=torch.zeros(2, 16))):
        with pytest.raises(ValueError):
            moe.gated_ffn_args(x, off, wg, wg, wd, **bad)
    for x2, off2, a, b, c in ((x[:, :8].contiguous(), off, wg, wg, wd), (x, off[:2], wg, wg, wd),
                              (x, off.long(), wg, wg, wd), (x, off, wg, wd, wd),
                              (x, off, wg, wg, wg), (x, off, wg.float(), wg, wd),
                              (x.t().contiguous().t(), off, wg, wg, wd), (x.half(), off, wg, wg, wd)):
        with pytest.raises(ValueError):
            moe.gated_ffn_args(x2, off2, a, b, c)
    g = torch.zeros(4)
    for bad in (lambda: moe.moe_grad_norm([]), lambda: moe.moe_grad_norm([g.double()]),
                lambda: moe.moe_clip_grads([g], torch.zeros(2), 1.0),
                lambda: moe.moe_clip_grads([g], torch.zeros(()).double(), 1.0),
                lambda: moe.moe_clip_grads([g], torch.zeros(()), 1.0, out=[]),
                lambda: moe.moe_clip_grads([g], torch.zeros(()), 1.0, out=[torch.zeros(3)]),
                lambda: moe.moe_clip_grads([torch.zeros(4, 4).t()[:2]], torch.zeros(()), 1.0)):
        with pytest.raises(ValueError):
            bad()
