"""GPU parity of the gated expert FFN (moe_gated_ffn, moe_gated_ffn_backward) with its definition
in 64 bits, within element-wise bounds on the arithmetic (tests/gated_ref.py)."""
import itertools

import pytest
import torch

from mixture_experts_layer_57_b200 import moe
from tests import gated_ref

pytestmark = pytest.mark.gpu
SENTINEL = 77.0
NAMES = ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down")


def make(E, counts, d, f, dtype, bias=True, seed=0, first=0, slack=3):
    """Inputs on the GPU. Rows outside every segment hold NaN, and so do the parameters of experts
    without rows: nothing there may reach an output."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=gen) * std).to(dtype)  # noqa: E731
    off = torch.tensor([first] + counts, dtype=torch.int64).cumsum(0).to(torch.int32)
    rows = int(off[-1]) + slack
    c = dict(x=rnd(rows, d), dy=rnd(rows, d), off=off.cuda(), counts=counts,
             w_gate=rnd(E, f, d, std=d ** -0.5), w_up=rnd(E, f, d, std=d ** -0.5),
             w_down=rnd(E, d, f, std=f ** -0.5))
    for n, k in (("b_gate", f), ("b_up", f), ("b_down", d)):
        c[n] = rnd(E, k, std=0.2) if bias else None
    for t in (c["x"], c["dy"]):
        t[:first] = float("nan")
        t[int(off[-1]):] = float("nan")
    for e, n in enumerate(counts):
        if n == 0:
            for k in NAMES:
                if c[k] is not None:
                    c[k][e] = float("nan")
    return c


def args_of(c, act="silu", out_dtype=None, hint=None):
    return moe.gated_ffn_args(c["x"], c["off"], *(c[n] for n in NAMES), act=act,
                              out_dtype=out_dtype or c["x"].dtype,
                              capacity_hint=max(c["counts"]) if hint is None else hint)


def run(c, act, out_dtype=None, grad_dtype=None, hint=None):
    """Forward and backward into sentinel-filled outputs."""
    x = c["x"]
    args = args_of(c, act, out_dtype, hint)
    y = torch.full(x.shape, SENTINEL, dtype=out_dtype or x.dtype, device="cuda")
    f = args.d_ff
    h = torch.full((x.shape[0], f), SENTINEL, dtype=x.dtype, device="cuda")
    saved = torch.full((2, x.shape[0], f), SENTINEL, dtype=x.dtype, device="cuda")
    r = moe.moe_gated_ffn(args, y_packed=y, h_packed=h, saved=saved)
    assert moe.moe_get_device_error(r["ws"]) == 0
    gd = grad_dtype or x.dtype
    ws = moe.workspace(moe.moe_gated_ffn_backward_workspace_bytes(args), "cuda")
    grads = {"d" + n: torch.full_like(c[n], SENTINEL, dtype=gd) for n in NAMES if c[n] is not None}
    grads["dx_packed"] = torch.full_like(y, SENTINEL)
    moe.moe_gated_ffn_backward(args, c["dy"], h, saved, grads, ws=ws)
    assert moe.moe_get_device_error(ws) == 0
    return dict(y=y, **grads), dict(h=h, saved=saved)


def compare(c, got, act, kept=None):
    """Every output against the definition; rows outside the segments still hold the sentinel."""
    a = int(c["off"][0])
    for e, n in enumerate(c["counts"]):
        params = {k: None if c[k] is None else c[k][e] for k in NAMES}
        if n == 0:
            for k in NAMES:
                if c[k] is not None:
                    assert bool((got["d" + k][e] == 0).all()), f"expert {e}: d{k} without rows"
            continue
        ref = gated_ref.segment(c["x"][a:a + n], params, act, c["dy"][a:a + n])
        for name in ("y", "dx_packed"):
            gated_ref.check(f"expert {e}: {name}", got[name][a:a + n], *ref[name])
        for k in NAMES:
            if c[k] is not None:
                gated_ref.check(f"expert {e}: d{k}", got["d" + k][e], *ref["d" + k])
        a += n
    outside = [got["y"], got["dx_packed"]] + ([] if kept is None else [kept["h"], *kept["saved"]])
    for t in outside:
        assert bool((t[:int(c["off"][0])] == SENTINEL).all()) and bool((t[a:] == SENTINEL).all())


BF16_SEGMENTS = [
    [1],                                  # a single token through a dense block
    [1, 0, 1, 1, 0, 1],                   # decoding: one row an expert, experts without rows
    [0, 0, 17],
    [20, 3, 0, 17, 32],
    [50, 64, 1, 0, 33],
    [128, 127, 0, 1, 100, 16],
    [300, 257, 0, 5, 256, 513],           # several wide tiles an expert
    [1000],
]


@pytest.mark.parametrize("counts", BF16_SEGMENTS, ids=str)
def test_bf16_segments(cuda_ok, counts):
    c = make(len(counts), counts, 256, 384, torch.bfloat16, seed=len(counts), first=2)
    got, kept = run(c, "silu")
    compare(c, got, "silu", kept)


@pytest.mark.parametrize("d,f", [(8, 8), (64, 8), (8, 200), (136, 264), (72, 1032), (1040, 24), (520, 1000)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_bf16_odd_widths(cuda_ok, d, f, act):
    c = make(3, [70, 0, 129], d, f, torch.bfloat16, seed=d + f)
    got, kept = run(c, act)
    compare(c, got, act, kept)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 33, 63, 65, 127, 129, 255, 257])
def test_bf16_dense_block_rows(cuda_ok, rows):
    c = make(1, [rows], 520, 776, torch.bfloat16, bias=False, seed=rows)
    got, kept = run(c, "silu")
    compare(c, got, "silu", kept)


@pytest.mark.parametrize("out_dtype,grad_dtype", list(itertools.product(
    [torch.float32, torch.bfloat16], [torch.float32, torch.bfloat16])))
def test_bf16_output_types(cuda_ok, out_dtype, grad_dtype):
    c = make(4, [5, 200, 0, 31], 128, 256, torch.bfloat16, seed=3)
    got, kept = run(c, "gelu", out_dtype, grad_dtype)
    compare(c, got, "gelu", kept)


@pytest.mark.parametrize("hint", [0, 1, 16, 40, 100, 200, 1 << 40])
def test_capacity_hint_may_be_wrong(cuda_ok, hint):
    c = make(3, [40, 0, 150], 128, 136, torch.bfloat16, seed=4)
    got, kept = run(c, "silu", hint=hint)
    compare(c, got, "silu", kept)


def test_bf16_wide_layer(cuda_ok):
    c = make(2, [129, 300], 2048, 4104, torch.bfloat16, bias=False, seed=5)
    got, kept = run(c, "silu")
    compare(c, got, "silu", kept)


def test_bf16_many_experts(cuda_ok):
    counts = [(7 * i) % 5 for i in range(1024)]
    c = make(1024, counts, 64, 64, torch.bfloat16, seed=6)
    got, kept = run(c, "silu")
    compare(c, got, "silu", kept)


@pytest.mark.parametrize("counts", [[16, 0, 7, 3], [1], [64], [200, 1, 0, 130]], ids=str)
@pytest.mark.parametrize("d,f", [(32, 64), (33, 131), (257, 77)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_fp32(cuda_ok, counts, d, f, act):
    c = make(len(counts), counts, d, f, torch.float32, seed=d, first=1)
    got, kept = run(c, act)
    compare(c, got, act, kept)


def test_fp32_large_tiles(cuda_ok):
    c = make(2, [1100, 900], 512, 1027, torch.float32, seed=8)
    got, kept = run(c, "silu")
    compare(c, got, "silu", kept)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_large_gates_saturate(cuda_ok, dtype):
    # gates far out on both sides: e^-z overflows, act is z or 0, act' is 1 or 0
    c = make(1, [40], 64, 128, dtype, bias=True, seed=9)
    c["b_gate"].copy_(torch.where(torch.arange(128, device="cuda") % 2 == 0, 300.0, -300.0))
    for act in ("silu", "gelu"):
        got, kept = run(c, act)
        compare(c, got, act, kept)


def test_other_experts_infinities_stay_theirs(cuda_ok):
    # infinite weights and rows of one expert reach no output of another
    c = make(3, [37, 20, 41], 72, 88, torch.bfloat16, bias=False, seed=10)
    clean, _ = run(c, "silu")
    a, b = 37, 57
    for n in ("w_gate", "w_up", "w_down"):
        c[n][1, 0] = float("inf")
        c[n][1, -1] = float("nan")
    c["x"][a:b] = float("inf")
    c["dy"][a:b] = float("-inf")
    got, _ = run(c, "silu")
    for n in ("y", "dx_packed"):
        assert torch.equal(got[n][:a], clean[n][:a]) and torch.equal(got[n][b:98], clean[n][b:98])
    for n in ("dw_gate", "dw_up", "dw_down"):
        assert torch.equal(got[n][::2], clean[n][::2])


def test_gradients_match_differences(cuda_ok):
    # the objective sum(dy * y) by central differences of the forward pass, fp32 layer
    c = make(2, [6, 9], 17, 23, torch.float32, seed=11, slack=0)
    got, _ = run(c, "gelu")

    def objective():
        y = moe.moe_gated_ffn(args_of(c, "gelu"))["y_packed"]
        return float((c["dy"].double() * y.double()).sum())

    gen = torch.Generator().manual_seed(1)
    eps = 2.0 ** -6
    for name, grad in [("x", "dx_packed")] + [(n, "d" + n) for n in NAMES]:
        t = c[name].view(-1)
        for i in torch.randint(t.numel(), (5,), generator=gen).tolist():
            keep = t[i].item()
            t[i] = keep + eps
            up, hi = objective(), t[i].item()
            t[i] = keep - eps
            down, lo = objective(), t[i].item()
            t[i] = keep
            # the third derivative's share (eps^2 times a few) and the objective's fp32 rounding
            assert abs((up - down) / (hi - lo) - got[grad].view(-1)[i].item()) <= 5e-3, (name, i)


def test_calls_repeat_bit_for_bit(cuda_ok):
    c = make(5, [1, 130, 0, 64, 300], 264, 520, torch.bfloat16, seed=12)
    one, _ = run(c, "silu")
    two, _ = run(c, "silu")
    for n in one:
        assert torch.equal(one[n], two[n]), n


def test_no_rows(cuda_ok):
    for dtype in (torch.float32, torch.bfloat16):
        c = make(3, [0, 0, 0], 64, 72, dtype, seed=13, slack=0)
        args = args_of(c, hint=0)
        r = moe.moe_gated_ffn(args, train=True)
        g = moe.moe_gated_ffn_backward(args, c["dy"], r["h_packed"], r["saved"], grad_dtype=dtype)
        for n in NAMES:
            assert bool((g["d" + n] == 0).all()), n


def test_bad_offsets_are_flagged(cuda_ok):
    for dtype in (torch.float32, torch.bfloat16):
        c = make(2, [8, 4], 64, 128, dtype, seed=14)
        c["off"] = torch.tensor([0, 8, 4], dtype=torch.int32, device="cuda")
        r = moe.moe_gated_ffn(args_of(c))
        assert moe.moe_get_device_error(r["ws"]) == 3   # MOE_DEVERR_BAD_OFFSETS
        c["off"] = torch.tensor([0, 8, 400], dtype=torch.int32, device="cuda")
        r = moe.moe_gated_ffn(args_of(c))
        assert moe.moe_get_device_error(r["ws"]) == 3


def test_other_stream_and_graph(cuda_ok):
    c = make(4, [33, 0, 150, 70], 136, 264, torch.bfloat16, seed=15)
    want, _ = run(c, "silu")
    s = torch.cuda.Stream()
    args = args_of(c)
    with torch.cuda.stream(s):
        s.wait_stream(torch.cuda.default_stream())
    r = moe.moe_gated_ffn(args, train=True, stream=s)
    g = moe.moe_gated_ffn_backward(args, c["dy"], r["h_packed"], r["saved"], grad_dtype=torch.bfloat16,
                                   stream=s)
    s.synchronize()
    n = sum(c["counts"])
    assert torch.equal(r["y_packed"][:n], want["y"][:n])
    assert torch.equal(g["dw_gate"], want["dw_gate"])
    # captured: the replay follows new inputs in place
    ws = moe.workspace(moe.moe_gated_ffn_backward_workspace_bytes(args), "cuda")
    y, h, saved = r["y_packed"], r["h_packed"], r["saved"]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.moe_gated_ffn(args, y_packed=y, h_packed=h, saved=saved, ws=ws)
        moe.moe_gated_ffn_backward(args, c["dy"], h, saved, g, ws=ws)
    c["x"].mul_(0.5)
    want, _ = run(c, "silu")
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[:n], want["y"][:n])
    assert torch.equal(g["dx_packed"][:n], want["dx_packed"][:n])
    for k in NAMES:
        assert torch.equal(g["d" + k], want["d" + k]), k


def test_gated_layer_from_router_to_combine(cuda_ok):
    """The entry points together, as a gated MoE layer is run: router, dispatch, gated experts,
    combine; then the experts' backward pass and clipping of their gradients."""
    T, d, f, E, k = 300, 128, 264, 6, 2
    gen = torch.Generator(device="cuda").manual_seed(16)
    rnd = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=gen) * std).to(torch.bfloat16)  # noqa: E731
    x = rnd(T, d)
    w_router = torch.randn(E, d, device="cuda", generator=gen) * 0.1
    w = dict(w_gate=rnd(E, f, d, std=0.1), w_up=rnd(E, f, d, std=0.1), w_down=rnd(E, d, f, std=0.1))
    r = moe.moe_router_topk(x, w_router, k)
    C = moe.moe_capacity(T, E, k, 1.0)
    p = moe.moe_dispatch(x, r["expert_ids"], E, C)
    args = moe.gated_ffn_args(p["x_packed"], p["expert_offsets"], w["w_gate"], w["w_up"], w["w_down"],
                              rows_max=p["rows_max"], capacity_hint=C)
    b = moe.moe_gated_ffn(args, train=True)
    out = moe.moe_combine(b["y_packed"], p["expert_offsets"], r["expert_ids"], p["slot"], r["gates"],
                          residual=x, out_dtype=torch.float32)["out"]
    ref, tol = x.double(), torch.zeros(T, d, dtype=torch.float64, device="cuda")
    n_drop = 0
    for j in range(k):
        for e in range(E):
            t = ((r["expert_ids"][:, j] == e) & (p["slot"][:, j] >= 0)).nonzero()[:, 0]
            y, bound = gated_ref.segment(x[t], {n: (v[e] if v is not None else None) for n, v in
                                                dict(w, b_gate=None, b_up=None, b_down=None).items()},
                                         "silu")["y"]
            g = r["gates"][t, j].double()[:, None]
            ref[t] += g * y
            tol[t] += g * bound
        n_drop += int((p["slot"][:, j] < 0).sum())
    assert n_drop > 0
    # the combine's k + 1 fp32 additions
    assert bool(((out.double() - ref).abs() <= tol + 2.0 ** -22 * (ref.abs() + 4)).all())
    dy = rnd(*p["x_packed"].shape)
    g = moe.moe_gated_ffn_backward(args, dy, b["h_packed"], b["saved"])
    names = ["dw_gate", "dw_up", "dw_down"]
    before = [g[n].double() for n in names]
    norm = moe.moe_clip_grad_norm([g[n] for n in names], 1.0)
    total = sum(float(t.square().sum()) for t in before) ** 0.5
    assert total > 1.0 and abs(norm.item() - total) <= 2.0 ** -19 * total
    for n, t in zip(names, before):
        assert bool(((g[n].double() - t / (total + 1e-6)).abs() <= 2.0 ** -19 * t.abs() / total).all()), n


@pytest.mark.parametrize("most", [1, 30, 64, 100, 200])
def test_bf16_many_feature_tiles(cuda_ok, most):
    # enough tiles to fill the device several times: pairs with two weight tiles up to 128 rows
    gen = torch.Generator().manual_seed(most)
    counts = torch.randint(most + 1, (40,), generator=gen).tolist()
    counts[3], counts[7] = 0, most
    c = make(40, counts, 520, 1032, torch.bfloat16, seed=most, first=1)
    got, kept = run(c, "gelu")
    compare(c, got, "gelu", kept)


@pytest.mark.parametrize("rows", [1, 5, 33, 64, 100, 128])
def test_bf16_dense_block_split_sums(cuda_ok, rows):
    # few tiles and long sums: every product is split over clusters
    c = make(1, [rows], 1024, 2056, torch.bfloat16, seed=rows)
    got, kept = run(c, "silu")
    compare(c, got, "silu", kept)


def test_bf16_small_and_large_scales(cuda_ok):
    # what the forward pass keeps has a range of its own: activations far from 1 on either side
    for std in (2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 40):
        c = make(2, [33, 60], 64, 72, torch.bfloat16, bias=False, seed=17)
        c["w_up"].mul_(std)
        got, kept = run(c, "silu")
        compare(c, got, "silu", kept)


def test_bf16_infinity_in_one_feature(cuda_ok):
    # an infinite up weight makes its feature's column infinite or NaN and no other
    c = make(1, [40], 64, 128, torch.bfloat16, bias=False, seed=18)
    clean, kept = run(c, "silu")
    c["w_up"][0, 5] = float("inf")
    got, bad = run(c, "silu")
    keep = torch.arange(128, device="cuda") != 5
    assert torch.equal(bad["h"][:40, keep], kept["h"][:40, keep])
    assert not bool(torch.isfinite(bad["h"][:40, 5]).any())
    # its neighbours share an exponent with it and keep 7 bits there: 2^-7 of each in their gradients
    near = keep & (torch.arange(128, device="cuda") < 8)
    far = torch.arange(128, device="cuda") >= 8
    assert torch.equal(got["dw_up"][0, far], clean["dw_up"][0, far])
    assert bool(torch.isfinite(got["dw_up"][0, near]).all())


@pytest.mark.parametrize("counts", [[1], [2], [3], [4], [5], [8], [1, 0, 2, 0, 1], [0, 0, 3, 4, 0, 1], [0, 1, 0]],
                         ids=str)
@pytest.mark.parametrize("dtype,d,f", [(torch.bfloat16, 264, 520), (torch.bfloat16, 8, 24),
                                       (torch.float32, 257, 77), (torch.float32, 33, 131)], ids=str)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_few_rows_forward(cuda_ok, counts, dtype, d, f, act):
    # without the saved tensors, as decoding runs it; rows before and behind the segments stay
    for first, slack in ((0, 0), (2, 1)):
        c = make(len(counts), counts, d, f, dtype, seed=d + len(counts), first=first, slack=slack)
        for out_dtype in {dtype, torch.float32}:
            y = torch.full(c["x"].shape, SENTINEL, dtype=out_dtype, device="cuda")
            r = moe.moe_gated_ffn(args_of(c, act, out_dtype), y_packed=y)
            assert moe.moe_get_device_error(r["ws"]) == 0
            a = first
            for e, n in enumerate(counts):
                if n:
                    params = {k: None if c[k] is None else c[k][e] for k in NAMES}
                    gated_ref.check(f"expert {e}: y", y[a:a + n],
                                    *gated_ref.segment(c["x"][a:a + n], params, act)["y"])
                a += n
            assert bool((y[:first] == SENTINEL).all()) and bool((y[a:] == SENTINEL).all())


def test_few_rows_bad_offsets(cuda_ok):
    for dtype in (torch.float32, torch.bfloat16):
        c = make(2, [2, 1], 64, 128, dtype, seed=19, slack=0)
        c["off"] = torch.tensor([0, 2, 1], dtype=torch.int32, device="cuda")
        y = torch.full(c["x"].shape, SENTINEL, dtype=dtype, device="cuda")
        r = moe.moe_gated_ffn(args_of(c), y_packed=y)
        assert moe.moe_get_device_error(r["ws"]) == 3
        assert bool((y == SENTINEL).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_tensor_for_both_projections(cuda_ok, dtype):
    c = make(2, [33, 150], 128, 272, dtype, seed=20)
    c["w_up"] = c["w_gate"]
    got, kept = run(c, "silu")
    compare(c, got, "silu", kept)


def test_up_weights_before_gate_weights(cuda_ok):
    # the projections in one allocation, in either order, and with a width off the 16-row groups
    for d, f in ((128, 272), (128, 264)):
        c = make(2, [33, 150], d, f, torch.bfloat16, seed=21)
        both = torch.empty(2, 2, f, d, dtype=torch.bfloat16, device="cuda")
        for order in (("w_gate", "w_up"), ("w_up", "w_gate")):
            e = dict(c)
            for i, n in enumerate(order):
                both[i].copy_(c[n])
                e[n] = both[i]
            got, kept = run(e, "gelu")
            compare(e, got, "gelu", kept)


def test_two_streams_at_once(cuda_ok):
    cases = [make(6, [40, 0, 130, 7, 64, 300], 264, 520, torch.bfloat16, seed=22),
             make(3, [100, 30, 1], 257, 131, torch.float32, seed=23)]
    want = [run(c, "silu")[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    out = []
    for _ in range(5):
        for c, s in zip(cases, streams):
            args = args_of(c)
            r = moe.moe_gated_ffn(args, train=True, stream=s)
            g = moe.moe_gated_ffn_backward(args, c["dy"], r["h_packed"], r["saved"],
                                           grad_dtype=c["x"].dtype, stream=s)
            out.append((r["y_packed"], g))
    torch.cuda.synchronize()
    for i, (y, g) in enumerate(out):
        w, n = want[i % 2], sum(cases[i % 2]["counts"])
        assert torch.equal(y[:n], w["y"][:n]) and torch.equal(g["dx_packed"][:n], w["dx_packed"][:n])
        for k in NAMES:
            assert torch.equal(g["d" + k], w["d" + k]), k


def test_stream_of_no_such_device_is_refused(cuda_ok):
    c = make(1, [4], 64, 72, torch.bfloat16, seed=24)

    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 7), 0

    with pytest.raises(ValueError):
        moe.moe_gated_ffn(args_of(c), stream=Elsewhere())
    with pytest.raises(ValueError):
        moe.moe_grad_norm([c["x"]], stream=Elsewhere())


@pytest.mark.parametrize("counts,d,f", [([700], 260, 1031), ([90, 0, 70, 100], 512, 1024),
                                        ([3, 30, 0, 64, 65], 700, 301)], ids=str)
def test_fp32_shapes_of_every_tile(cuda_ok, counts, d, f):
    # tiles of 128 and of 64 rows and split sums, rows on and off 16-byte boundaries
    c = make(len(counts), counts, d, f, torch.float32, seed=d, first=3)
    got, kept = run(c, "gelu")
    compare(c, got, "gelu", kept)


def test_fp32_largest_and_smallest_factors(cuda_ok):
    # the two-part split neither overflows near fp32's largest value nor loses small factors: with the
    # rows and the weights of the first products scaled by inverse powers of two, every part of every
    # factor scales with it (the least bits, below 2^-40 here, stay above 2^-126), so the results are
    # the same bits
    c = make(1, [20], 64, 64, torch.float32, bias=False, seed=25, slack=0)
    clean = moe.moe_gated_ffn(args_of(c), train=True)["y_packed"].clone()
    for scale in (2.0 ** 80, 2.0 ** -80):
        e = dict(c, x=c["x"] / scale, w_gate=c["w_gate"] * scale, w_up=c["w_up"] * scale)
        y = moe.moe_gated_ffn(args_of(e), train=True)["y_packed"]
        assert torch.equal(y[:20], clean[:20]), scale
    c["x"][0, 0] = torch.finfo(torch.float32).max
    c["w_gate"][0, :, 0] = 2.0 ** -126
    c["w_up"][0, :, 0] = 2.0 ** -126
    h = moe.moe_gated_ffn(args_of(c), train=True)["h_packed"]
    assert bool(torch.isfinite(h[0]).all())


def test_fp32_many_experts(cuda_ok):
    counts = [(5 * i) % 4 for i in range(1024)]
    c = make(1024, counts, 33, 17, torch.float32, seed=26)
    got, kept = run(c, "silu")
    compare(c, got, "silu", kept)


def test_few_rows_of_many_experts(cuda_ok):
    counts = [0] * 1024
    counts[0], counts[517], counts[1023] = 2, 1, 3
    c = make(1024, counts, 33, 17, torch.float32, seed=27, slack=0)
    y = moe.moe_gated_ffn(args_of(c))["y_packed"]
    a = 0
    for e in (0, 517, 1023):
        n = counts[e]
        params = {k: c[k][e] for k in NAMES}
        gated_ref.check("y", y[a:a + n], *gated_ref.segment(c["x"][a:a + n], params, "silu")["y"])
        a += n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_long_segment(cuda_ok, dtype):
    c = make(3, [3, 70_001, 20], 40, 24, dtype, seed=28)
    got, kept = run(c, "gelu")
    compare(c, got, "gelu", kept)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 64), (torch.float32, 17)], ids=str)
def test_hidden_tensors_past_32_bit_offsets(cuda_ok, dtype, d):
    # h, saved, dg and du have more than 2^31 elements; the last expert lies behind that
    rows, last, f = 262_300, 100, 8192
    c = make(2, [rows, last], d, f, dtype, bias=False, seed=29, slack=0)
    assert (rows + last) * f > 2 ** 31 and rows * f > 2 ** 31
    args = args_of(c)
    r = moe.moe_gated_ffn(args, train=True)
    g = moe.moe_gated_ffn_backward(args, c["dy"], r["h_packed"], r["saved"], grad_dtype=dtype)
    ref = gated_ref.segment(c["x"][rows:], {k: None if c[k] is None else c[k][1] for k in NAMES}, "silu",
                            c["dy"][rows:])
    gated_ref.check("y", r["y_packed"][rows:], *ref["y"])
    gated_ref.check("dx", g["dx_packed"][rows:], *ref["dx_packed"])
    for k in ("w_gate", "w_up", "w_down"):
        gated_ref.check("d" + k, g["d" + k][1], *ref["d" + k])
    # and rows on both sides of the border, of the first expert
    at = 2 ** 31 // f - 20
    ref = gated_ref.segment(c["x"][at:at + 40], {k: None if c[k] is None else c[k][0] for k in NAMES}, "silu",
                            c["dy"][at:at + 40])
    gated_ref.check("y", r["y_packed"][at:at + 40], *ref["y"])
    gated_ref.check("dx", g["dx_packed"][at:at + 40], *ref["dx_packed"])
