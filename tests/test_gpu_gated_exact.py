"""The gated FFN on whole numbers, forward and backward, bit for bit.

Gates of 20 or more saturate: act(z) is z and act'(z) is 1 in fp32 arithmetic. With x, dy and the
weights in {-1, 0, 1} and whole biases every product and every partial sum is then a whole number below
2^24, exact in fp32 in any order, and the roundings of h, du and dg to bf16 are known. So a row, a block
of K or a part of a split sum that is lost, counted twice or taken from elsewhere shows, however long
the sum."""
import pytest
import torch

from mixture_experts_layer_57_b200 import moe

pytestmark = pytest.mark.gpu
SENTINEL = 77.0
PARAMS = ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down")


def signs(gen, shape, p, dtype):
    u = torch.rand(shape, device="cuda", generator=gen)
    return ((u < p / 2).to(dtype) - (u > 1 - p / 2).to(dtype))


def make(counts, d, f, dtype, seed, first=0, slack=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E = len(counts)
    off = torch.tensor([first] + counts).cumsum(0).to(torch.int32)
    rows = int(off[-1]) + slack
    some = min(0.25, 8 / d)   # few terms a row: sums of x and of dy stay small at any width
    c = dict(counts=counts, off=off.cuda(), x=signs(gen, (rows, d), some, dtype),
             dy=signs(gen, (rows, d), some, dtype))
    for n, shape in (("w_gate", (E, f, d)), ("w_up", (E, f, d)), ("w_down", (E, d, f))):
        c[n] = signs(gen, shape, 0.5, dtype)
    c["b_gate"] = torch.randint(64, 96, (E, f), device="cuda", generator=gen).to(dtype)
    c["b_up"] = torch.randint(-2, 3, (E, f), device="cuda", generator=gen).to(dtype)
    c["b_down"] = torch.randint(-9, 10, (E, d), device="cuda", generator=gen).to(dtype)
    for t in (c["x"], c["dy"]):
        t[:first] = float("nan")
        t[int(off[-1]):] = float("nan")
    return c


def run(c, act, grad_dtype, out_dtype, hint=None):
    x = c["x"]
    args = moe.gated_ffn_args(x, c["off"], *(c[n] for n in PARAMS), act=act, out_dtype=out_dtype,
                              capacity_hint=max(c["counts"]) if hint is None else hint)
    y = torch.full(x.shape, SENTINEL, dtype=out_dtype, device="cuda")
    r = moe.moe_gated_ffn(args, y_packed=y, train=True)
    assert moe.moe_get_device_error(r["ws"]) == 0
    grads = {"d" + n: torch.full_like(c[n], SENTINEL, dtype=grad_dtype) for n in PARAMS}
    grads["dx_packed"] = torch.full_like(y, SENTINEL)
    ws = moe.workspace(moe.moe_gated_ffn_backward_workspace_bytes(args), "cuda")
    moe.moe_gated_ffn_backward(args, c["dy"], r["h_packed"], r["saved"], grads, ws=ws)
    assert moe.moe_get_device_error(ws) == 0
    return dict(y=y, **grads)


def whole(*factors):
    """The product of matrices of whole numbers, none of whose partial sums can reach 2^24."""
    a, b = factors
    assert float((a.abs() @ b.abs()).max() if a.numel() and b.numel() else 0) < 2 ** 24
    return a @ b


def expect(c, e, rows):
    """What expert e gives for its rows, in fp64, rounded where the bf16 layer rounds."""
    x, dy = c["x"][rows].double(), c["dy"][rows].double()
    wg, wu, wd, bg, bu, bd = (c[n][e].double() for n in PARAMS)
    cut = lambda t: t.to(c["x"].dtype).double()  # noqa: E731
    zg, zu = whole(x, wg.T) + bg, whole(x, wu.T) + bu
    assert float(zg.min()) >= 20
    h = cut(zg * zu)
    dh = whole(dy, wd)
    du, dg = cut(dh * zg), cut(dh * zu)
    out = dict(y=whole(h, wd.T) + bd, dx_packed=whole(torch.cat([dg, du], 1), torch.cat([wg, wu])),
               dw_down=whole(dy.T, h), dw_gate=whole(dg.T, x), dw_up=whole(du.T, x))
    for n, t in (("db_gate", dg), ("db_up", du), ("db_down", dy)):
        assert float(t.abs().sum(0).max()) < 2 ** 24
        out[n] = t.sum(0)
    return out


def check(c, got):
    a = int(c["off"][0])
    for e, n in enumerate(c["counts"]):
        if n == 0:
            for k in PARAMS:
                assert bool((got["d" + k][e] == 0).all()), (e, k)
            continue
        want = expect(c, e, slice(a, a + n))
        for k in ("y", "dx_packed"):
            assert torch.equal(got[k][a:a + n], want[k].to(got[k].dtype)), (e, k)
        for k in PARAMS:
            assert torch.equal(got["d" + k][e], want["d" + k].to(got["d" + k].dtype)), (e, k)
        a += n
    for k in ("y", "dx_packed"):
        assert bool((got[k][:int(c["off"][0])] == SENTINEL).all()) and bool((got[k][a:] == SENTINEL).all())


SEGMENTS = [[1], [3, 0, 17, 64], [100, 16, 129, 0, 255], [300, 257, 513], [1000]]


@pytest.mark.parametrize("counts", SEGMENTS, ids=str)
@pytest.mark.parametrize("dtype,d,f", [(torch.bfloat16, 8, 24), (torch.bfloat16, 136, 264),
                                       (torch.bfloat16, 520, 1032), (torch.float32, 33, 131),
                                       (torch.float32, 260, 520)], ids=str)
def test_segments(cuda_ok, counts, dtype, d, f):
    c = make(counts, d, f, dtype, seed=d + len(counts), first=2, slack=1)
    check(c, run(c, "silu", torch.float32, dtype))
    check(c, run(c, "gelu", dtype, torch.float32))


@pytest.mark.parametrize("rows", [1, 33, 100, 128, 200])
def test_split_sums(cuda_ok, rows):
    c = make([rows], 1024, 2056, torch.bfloat16, seed=rows)
    check(c, run(c, "silu", torch.float32, torch.float32))


def test_many_feature_tiles(cuda_ok):
    counts = [(37 * i) % 131 for i in range(40)]
    c = make(counts, 520, 1032, torch.bfloat16, seed=5)
    check(c, run(c, "silu", torch.bfloat16, torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [4099, 40_000])
def test_long_segment(cuda_ok, dtype, rows):
    # thousands of K blocks and every split of the bias sums
    c = make([3, rows, 20], 40, 24, dtype, seed=rows)
    got = run(c, "silu", torch.float32, dtype)
    check(c, got)
    # what would go unnoticed within a bound that grows with the rows does not here
    want = expect(c, 1, slice(3, 3 + rows))
    for k in PARAMS:
        t = got["d" + k][1].double()
        assert not torch.equal(t, torch.zeros_like(t)) and torch.equal(t, want["d" + k])
    less = expect(c, 1, slice(3, 3 + rows - 16))
    assert all(not torch.equal(less["d" + k], want["d" + k]) for k in PARAMS)


@pytest.mark.parametrize("d,f", [(64, 272), (8, 608), (128, 48), (520, 1040)])
@pytest.mark.parametrize("between", ["none", "rows of a group", "one row", "ends of allocations"])
@pytest.mark.parametrize("order", [("w_gate", "w_up"), ("w_up", "w_gate")], ids=str)
def test_places_of_the_projections(cuda_ok, d, f, between, order):
    # the two weights side by side, at distances on and off whole groups of 16 rows, and each at the end of
    # an allocation of its own, behind which memory need not be mapped
    c = make([5, 0, 70, 33], d, f, torch.bfloat16, seed=d + f)
    n = 4 * f * d
    if between == "ends of allocations":
        torch.cuda.empty_cache()
        keep = [torch.empty(12 << 20, dtype=torch.bfloat16, device="cuda") for _ in order]
        w = {k: s[-n:].view(4, f, d) for k, s in zip(order, keep)}
    else:
        gap = {"none": 0, "rows of a group": 16 * d, "one row": d}[between]
        space = torch.full((2 * n + gap,), float("nan"), dtype=torch.bfloat16, device="cuda")
        w = {order[0]: space[:n].view(4, f, d), order[1]: space[n + gap:].view(4, f, d)}
    for k in order:
        w[k].copy_(c[k])
    e = dict(c, **w)
    check(e, run(e, "silu", torch.float32, torch.bfloat16))
