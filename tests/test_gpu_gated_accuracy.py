"""Accuracy of the gated FFN's activations where the element-wise bounds of whole products are too
wide to tell: pre-activations are set exactly through the biases (all weights of the first products are
zero), so the kept tensors and h show the activation alone."""
import math

import pytest
import torch

from mixture_experts_layer_57_b200 import moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def block(z, zu, dtype, act, rows=9, train=True):
    """One dense block whose rows all have the pre-activations z and zu [f]: h and the saved planes."""
    f, d = z.numel(), 8
    zero = torch.zeros(1, f, d, dtype=dtype, device="cuda")
    x = torch.ones(rows, d, dtype=dtype, device="cuda")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    args = moe.gated_ffn_args(x, off, zero, zero, torch.zeros(1, d, f, dtype=dtype, device="cuda"),
                              b_gate=z.to(dtype)[None].cuda(), b_up=zu.to(dtype)[None].cuda(), act=act)
    r = moe.moe_gated_ffn(args, train=train)
    h = r["h_packed"]
    assert all(torch.equal(h[0], h[i]) for i in range(rows))
    return h[0].double().cpu(), None if r["saved"] is None else r["saved"][:, rows - 1].cpu()


def exact(z, act):
    """act(z) and act'(z) in 64 bits without cancellation, with bounds on the relative error of an fp32
    evaluation. GeLU: the argument of erfc is off by 1.3 2^-24 of itself (a product and the constant),
    which erfc magnifies by at most z^2 + 1; erfc itself by 4 units (8 2^-24), the exponential of the
    density by 2 units after z^2 / 2 2^-24 from its argument; products and sums 2^-24 each. SiLU: the
    exponential, an addition, a division and a product."""
    z = z.double()
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        pdf = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        rc = ((z * z + 2) * 1.3 + 9) * U
        return (z * cdf, z.abs() * cdf * (rc + U), cdf + z * pdf,
                cdf * rc + (z * pdf).abs() * (z * z / 2 + 7) * U + (cdf + z * pdf).abs() * U)
    s = torch.sigmoid(z)
    t = 1 + z * torch.sigmoid(-z)
    return (z * s, 8 * U * (z * s).abs(), s * t,
            s * (z.abs() * (6 * s + 2 * torch.sigmoid(-z)) + 8 * t.abs()) * U)


def assert_within(got, want, bound, what):
    err = (got - want).abs()
    i = int((err / bound).argmax())
    assert bool((err <= bound).all()), f"{what}: {float(err[i]):.3g} of {float(want[i]):.6g}, " \
                                       f"{float(err[i] / bound[i]):.3g} times the bound, at {i}"


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_fp32_activation_and_derivative(cuda_ok, act):
    z = torch.linspace(-8, 8, 2049)
    a, ea, da, eda = exact(z, act)
    one = torch.ones_like(z)
    h, saved = block(z, one, torch.float32, act)
    for got in (h, saved[0].double(), block(z, one, torch.float32, act, rows=3, train=False)[0]):
        assert_within(got, a, ea + 2.0 ** -140, "act")
    assert_within(saved[1].double(), da, eda + 2.0 ** -140, "act'")


@pytest.mark.parametrize("act,far", [("silu", 80.0), ("gelu", 12.5)])
def test_bf16_activation(cuda_ok, act, far):
    # h is act(z) rounded once: half a step, and what the approximate exponential adds (its error is
    # 2 + 1.2 |argument| units, the argument's own rounding |argument| units: 2^-15 at either end here)
    z = torch.linspace(-far, far, 4096).to(torch.bfloat16).float()
    a = exact(z, act)[0]
    h, _ = block(z, torch.ones_like(z), torch.bfloat16, act)
    assert_within(h, a, (2.0 ** -8 + 2.0 ** -14) * a.abs() + 2.0 ** -133, "act")


def unpack(saved):
    """Eight neighbours of 16 bits with their shared code in bit 14 of each: bits 0..6 of it are half
    the exponent (rounded up), bit 7 says bf16 instead of fp16; 127: the top bits of each value itself."""
    w = saved.view(torch.int16).to(torch.int32).reshape(-1, 8) & 0xffff
    flag = (w >> 14) & 1
    code = sum(flag[:, 2 * i] << i | flag[:, 2 * i + 1] << (4 + i) for i in range(4))
    w = w & 0xbfff
    half, wide = code & 127, (code >> 7) == 1
    as16 = lambda t: torch.where(t >= 2 ** 15, t - 2 ** 16, t).to(torch.int16)  # noqa: E731
    fp16 = as16(w).view(torch.float16).double()
    bf16 = as16(w).view(torch.bfloat16).double()
    own = ((w & 0x8000) << 16 | (w & 0x3fff) << 17)
    own = torch.where(own >= 2 ** 31, own - 2 ** 32, own).to(torch.int32).view(torch.float32).double()
    v = torch.where(wide[:, None], bf16, fp16) * torch.exp2(2.0 * half - 126)[:, None].double()
    return torch.where((half == 127)[:, None], own, v).reshape(-1)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_saved_tensors_keep_eleven_bits(cuda_ok, act):
    gen = torch.Generator().manual_seed(1)
    z = (2 * torch.randn(4096, generator=gen)).to(torch.bfloat16).float()
    zu = torch.randn(4096, generator=gen).to(torch.bfloat16).float()
    a, _, da, _ = exact(z, act)
    q = zu.double() * da
    _, saved = block(z, zu, torch.bfloat16, act)
    for got, want, slack, what in ((unpack(saved[0]), a, 2.0 ** -16 * a.abs(), "act"),
                                   (unpack(saved[1]), q, 2.0 ** -18 * zu.double().abs(), "zu act'")):
        most = want.abs().reshape(-1, 8).max(1, keepdim=True).values.expand(-1, 8).reshape(-1)
        # half a step of 11 bits; values far below the block's largest: half of fp16's least step at a
        # scale that is at most four times the largest
        bound = 2.0 ** -11 * want.abs() + 2.0 ** -23 * most + slack
        # a block with a value below 2^-17, at a scale where its largest is 1/4 to 1, keeps 8 bits of each:
        # so may those with a ratio below 2^-15 (of GeLU gates this far out one in six)
        least = want.abs().reshape(-1, 8).min(1, keepdim=True).values.expand(-1, 8).reshape(-1)
        few = least < 2.0 ** -15 * most
        bound = torch.where(few, 2.0 ** -8 * want.abs() + slack, bound)
        assert_within(got, want, bound, what)
        # a plain bf16 copy is not as good
        assert float(((want.to(torch.bfloat16).double() - want).abs() > bound).double().mean()) > 0.2


@pytest.mark.parametrize("act,dead", [("silu", -20.0), ("gelu", -5.5)])
def test_saved_tensors_keep_small_values_beside_large_ones(cuda_ok, act, dead):
    # a feature whose gate is shut, among features whose gates are wide open: its gradients keep bf16's
    # 8 bits (one rounding of the kept value, one of du or dg)
    f, d, rows = 64, 8, 1
    z = torch.full((f,), 200.0)
    z[::8] = dead
    zu = torch.full((f,), 1024.0)
    zu[3::8] = 0.0
    one = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    zero = torch.zeros(1, f, d, dtype=torch.bfloat16, device="cuda")
    w_down = torch.zeros(1, d, f, dtype=torch.bfloat16, device="cuda")
    w_down[0, 0] = 1.0
    args = moe.gated_ffn_args(one(rows, d), torch.tensor([0, rows], dtype=torch.int32, device="cuda"), zero,
                              zero, w_down, b_gate=z.to(torch.bfloat16)[None].cuda(),
                              b_up=zu.to(torch.bfloat16)[None].cuda(), act=act)
    r = moe.moe_gated_ffn(args, train=True)
    g = moe.moe_gated_ffn_backward(args, one(rows, d), r["h_packed"], r["saved"])
    a, _, da, _ = exact(z, act)
    for name, want in (("dw_up", a), ("dw_gate", zu.double() * da)):
        got = g[name][0].double().cpu()
        for j in range(d):
            assert_within(got[:, j], want, (2 * 2.0 ** -8 + 2.0 ** -14) * want.abs() + 1e-300, name)


def test_saved_tensors_beside_a_magnitude_past_the_scale(cuda_ok):
    # a value of 2^126 or more, or an infinity: its seven neighbours keep the sign, the exponent and six
    # bits of mantissa of their own, cut (up to 2^-6 of the value)
    gen = torch.Generator().manual_seed(2)
    z = (2 * torch.randn(512, generator=gen)).to(torch.bfloat16).float()
    zu = (torch.randn(512, generator=gen) * 2.0 ** 20).to(torch.bfloat16).float()
    big = torch.arange(512) % 8 == 3
    a, _, da, _ = exact(z, "silu")
    for value in (3e38, 2.0 ** 126, float("inf")):
        zu[big] = value
        _, saved = block(z, zu, torch.bfloat16, "silu")
        q, want = unpack(saved[1]), zu.double() * da
        assert_within(q[~big], want[~big], (2.0 ** -6 + 2.0 ** -16) * want[~big].abs()
                      + zu.double().abs()[~big] * 2.0 ** -18, "neighbours")
        if value == float("inf"):
            assert bool((q[big] == want[big]).all())
        else:
            near = want[big].abs() >= 2.0 ** 126
            assert_within(q[big][near], want[big][near], 2.0 ** -5.9 * want[big][near].abs(), "large")
        assert_within(unpack(saved[0]), a, 2.0 ** -7.9 * a.abs(), "act")


def test_fp32_nan_of_any_payload(cuda_ok):
    # NaNs whose payload lies in the low bits only: the two-part split may not turn them into infinities
    # (second parts of the weights have the first ones' sign, so infinities would not cancel)
    for bits in (0x7f800001, 0x7f801fff, 0x7fc00000, 0x7fffffff, -1, -0x7fffff):
        x = torch.zeros(20, 32, device="cuda")
        x.view(torch.int32)[4, 7] = bits
        w = torch.full((1, 32, 32), 1 + 2.0 ** -13, device="cuda")
        args = moe.gated_ffn_args(x, torch.tensor([0, 20], dtype=torch.int32, device="cuda"), w, w, w)
        r = moe.moe_gated_ffn(args, train=True)
        for t in (r["h_packed"], r["y_packed"], r["saved"][0]):
            assert bool(torch.isnan(t[4]).all()), hex(bits & 0xffffffff)
            assert bool((t[:4] == 0).all()) and bool((t[5:] == 0).all())
