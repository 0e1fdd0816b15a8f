"""GPU parity of the gradient norm and of clipping with 64-bit sums.

Bounds: a thread's fp32 sum of at most 34 squares (32 of a chunk and an end on each side) is
within 35 * 2^-24 of its value, the sums above it are doubles, so the norm is within 18 * 2^-24 and
its rounding 2^-24; the factor adds four fp32 roundings, the output its own."""
import pytest
import torch

from mixture_experts_layer_57_b200 import moe

pytestmark = pytest.mark.gpu
NORM_TOL = 19 * 2.0 ** -24
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def make(sizes, dtypes, seed=0, std=1.0, offset=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n + offset, device="cuda", generator=gen) * std
        out.append(t.to(dtypes[i % len(dtypes)])[offset:])
    return out


def exact_norm(grads):
    return sum(float(g.double().square().sum()) for g in grads) ** 0.5


def check(grads, max_norm, out=None):
    before = [g.double() for g in grads]
    want = exact_norm(grads)
    norm = moe.moe_clip_grad_norm(grads, max_norm, out=out)
    assert abs(norm.item() - want) <= NORM_TOL * want
    k = min(1.0, max_norm / (want + 1e-6))
    for b, o in zip(before, grads if out is None else out):
        tol = (NORM_TOL + 5 * 2.0 ** -24 + STEP[o.dtype]) * (b * k).abs() + 2.0 ** -133
        assert bool(((o.double() - b * k).abs() <= tol).all())
    return norm


SIZES = [1, 7, 8, 255, 4096, 8191, 8192, 8193, 100_003]


@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], [torch.bfloat16, torch.float32]],
                         ids=str)
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 8])
def test_in_place(cuda_ok, dtypes, offset):
    check(make(SIZES, dtypes, seed=offset, offset=offset), 0.5)


@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dst", [torch.float32, torch.bfloat16])
def test_into_a_flat_buffer(cuda_ok, src, dst):
    grads = make(SIZES, [src], seed=1)
    total = sum(SIZES)
    flat = torch.full((total + 2,), 77.0, dtype=dst, device="cuda")
    keep = [g.clone() for g in grads]
    check(grads, 0.1, out=list(flat[1:-1].split(SIZES)))
    assert flat[0].item() == 77.0 and flat[-1].item() == 77.0
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))


@pytest.mark.parametrize("n", [1, 31, 48, 49, 1024, 1025, 2500])
def test_list_lengths(cuda_ok, n):
    check(make([1 + (37 * i) % 301 for i in range(n)], [torch.float32, torch.bfloat16], seed=n), 0.25)


def test_single_element_and_empty_tensors(cuda_ok):
    for sizes in ([1], [0, 1, 0], [0, 0, 5, 0]):
        check(make(sizes, [torch.float32], seed=2), 1e-3)
    norm = moe.moe_grad_norm(make([0, 0], [torch.float32]))
    assert norm.item() == 0.0


def test_large_tensor(cuda_ok):
    check(make([70_000_001, 3], [torch.bfloat16], seed=3, std=1e-3), 0.01)


def test_below_the_limit_nothing_changes(cuda_ok):
    for dtype in (torch.float32, torch.bfloat16):
        grads = make(SIZES, [dtype], seed=4)
        keep = [g.clone() for g in grads]
        out = [torch.empty_like(g) for g in grads]
        moe.moe_clip_grad_norm(grads, 1e9)
        moe.moe_clip_grad_norm(grads, 1e9, out=out)
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(grads, keep, out))


def test_limit_of_zero(cuda_ok):
    grads = make(SIZES, [torch.float32], seed=5)
    moe.moe_clip_grad_norm(grads, 0.0)
    assert all(bool((g == 0).all()) for g in grads)


@pytest.mark.parametrize("std", [1e-38, 1e-30, 1e-22, 1e-15, 1e10, 1e18, 1e25, 1e34])
def test_sizes_whose_squares_leave_fp32(cuda_ok, std):
    for dtype in (torch.float32, torch.bfloat16):
        grads = make([1000, 9001], [dtype], seed=6, std=std)
        want = exact_norm(grads)
        assert abs(moe.moe_grad_norm(grads).item() - want) <= NORM_TOL * want + 2.0 ** -149


def test_mixed_magnitudes(cuda_ok):
    grads = [torch.tensor([1e-25] * 50 + [3e20], device="cuda"), torch.tensor([4e20], device="cuda")]
    assert abs(moe.moe_grad_norm(grads).item() - 5e20) <= NORM_TOL * 5e20


def test_infinities_and_nan(cuda_ok):
    a = make([5000, 9000], [torch.float32], seed=7)
    a[1][8500] = float("inf")
    keep = [t.clone() for t in a]
    norm = moe.moe_clip_grad_norm(a, 1.0)
    assert norm.item() == float("inf")
    # a factor of zero: finite gradients become zero, the infinite one NaN
    assert bool((a[0] == 0).all()) and bool(torch.isnan(a[1][8500])) and bool((a[1][:8500] == 0).all())
    keep[0][3] = float("nan")
    assert torch.isnan(moe.moe_clip_grad_norm(keep, 1.0))
    assert all(bool(torch.isnan(t).all()) for t in keep)


def test_repeats_bit_for_bit_and_the_workspace_is_reusable(cuda_ok):
    grads = make([3_000_001, 17, 40_000], [torch.float32], seed=8)
    ws = moe.workspace(moe.moe_grad_norm_workspace_bytes(), "cuda")
    first = moe.moe_grad_norm(grads, ws=ws).clone()
    for _ in range(5):
        assert torch.equal(moe.moe_grad_norm(grads, ws=ws), first)
        moe.moe_grad_norm(grads[1:], ws=ws)


def test_graph_and_stream(cuda_ok):
    grads = make(SIZES, [torch.float32], seed=9)
    out = [torch.empty_like(g) for g in grads]
    norm = torch.empty((), device="cuda")
    ws = moe.workspace(moe.moe_grad_norm_workspace_bytes(), "cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    moe.moe_clip_grad_norm(grads, 0.5, out=out, norm=norm, ws=ws, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.moe_clip_grad_norm(grads, 0.5, out=out, norm=norm, ws=ws)
    for g in grads:
        g.mul_(3.0)
    want = [torch.empty_like(g) for g in grads]
    wnorm = moe.moe_clip_grad_norm(grads, 0.5, out=want)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, wnorm)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dst", [torch.float32, torch.bfloat16])
def test_places_of_any_relative_alignment(cuda_ok, src, dst):
    # gradient and output start at every distance from a 16-byte boundary, with lengths around the
    # vectors' and chunks' ends
    for a in range(8):
        for b in range(8):
            sizes = [1 + (5 * a + 3 * b) % 40, 61 + a, 8200 + 7 * b]
            grads = make([n + a for n in sizes], [src], seed=8 * a + b)
            grads = [g[a:] for g in grads]
            space = [torch.full((n + b + 3,), 77.0, dtype=dst, device="cuda") for n in sizes]
            check(grads, 0.5, out=[s[b:b + n] for s, n in zip(space, sizes)])
            for s, n in zip(space, sizes):
                assert bool((s[:b] == 77.0).all()) and bool((s[b + n:] == 77.0).all())


def test_tensor_past_32_bit_offsets(cuda_ok):
    n = 2 ** 31 + 9
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[0], g[-1] = 4.0, -8.0
    want = ((n - 2) * 0.25 + 16 + 64) ** 0.5
    norm = moe.moe_clip_grad_norm([g], want / 2)
    assert abs(norm.item() - want) <= NORM_TOL * want
    # the factor is 1/2 within a few 2^-24, and bf16 rounds these products to exact halves
    assert g[0].item() == 2.0 and g[-1].item() == -4.0
    assert g[1].item() == 0.25 and bool((g[-1000:-1] == 0.25).all()) and bool((g[2 ** 31 - 500:2 ** 31] == 0.25).all())
