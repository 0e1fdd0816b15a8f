"""Cases of the gated feed-forward block and of gradient clipping, with their plain forms.

Three operators, each in the plain form (elementary torch operations in 32 bits) and as the calls
a user makes of the library:

* ``ffn``    the gated block forward on expert-major rows: for every row r of expert e
             h = act(W_gate[e] x + b_gate[e]) * (W_up[e] x + b_up[e]),  y = W_down[e] h + b_down[e]
* ``train``  the same forward keeping its state, then the backward pass: from dy the gradients of
             the rows, the three weights and the biases
* ``clip``   the global 2-norm of a list of gradients, and the gradients times
             min(1, max_norm / (norm + 1e-6)) written to a flat buffer

Sizes are the library's own workloads (the GPT-350M and GPT-1.3B MoE layers, the top-2 layer of 8
experts, decode, the tiny fp32 layer), odd ones around them, and a dense block (one expert that
takes every row).
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token through a dense gated block of the 1.3B shape: the latency of a decode step
        dict(name="ffn-token", op="ffn", dtype="bf16", E=1, rows=1, d=2048, f=8192, act="silu",
             bias=False, spread="even", factor=1.0, mix=1),
        # 32 decoding sequences over 128 experts: weights of the touched experts stream from HBM
        dict(name="ffn-decode-e128", op="ffn", dtype="bf16", E=128, rows=32, d=2048, f=8192,
             act="silu", bias=False, spread="even", factor=8.0, mix=2),
        # prefill of the 350M layer, 128 rows an expert on average, with biases and GeLU gates
        dict(name="ffn-gpt350m-e128", op="ffn", dtype="bf16", E=128, rows=16384, d=1024, f=4096,
             act="gelu", bias=True, spread="even", factor=1.25, mix=3),
        # prefill of the top-2 layer of 8 large experts under a Zipf load: bound by the products
        dict(name="ffn-top2-e8", op="ffn", dtype="bf16", E=8, rows=16384, d=4096, f=14336,
             act="silu", bias=False, spread="zipf", factor=1.25, mix=4),
        # fp32 layer of odd sizes, as the library's fp32 checks use
        dict(name="ffn-f32-odd", op="ffn", dtype="f32", E=4, rows=1000, d=501, f=1334, act="silu",
             bias=True, spread="even", factor=2.0, mix=5),
        # one training step of the 350M layer's experts: gradients of every weight are written
        dict(name="train-gpt350m-e128", op="train", dtype="bf16", E=128, rows=16384, d=1024,
             f=4096, act="silu", bias=False, spread="even", factor=1.25, mix=6),
        # a small ragged training step: sizes off every tile, experts without rows, biases
        dict(name="train-ragged", op="train", dtype="bf16", E=17, rows=1999, d=1032, f=2744,
             act="gelu", bias=True, spread="zipf", factor=3.0, mix=7),
        # one training step of the top-2 layer: bound by the products
        dict(name="train-top2-e8", op="train", dtype="bf16", E=8, rows=16384, d=4096, f=14336,
             act="silu", bias=False, spread="zipf", factor=1.25, mix=8),
        # an fp32 training step of odd sizes
        dict(name="train-f32-odd", op="train", dtype="f32", E=3, rows=777, d=321, f=1027,
             act="silu", bias=True, spread="even", factor=2.0, mix=9),
        # the gradients of a tiny model: latency of the two passes
        dict(name="clip-small", op="clip", dtype="f32", to="f32", tensors=24, total=200_000,
             clip=0.5, mix=10),
        # fp32 gradients of a dense 350M model, some 300 tensors
        dict(name="clip-dense350m", op="clip", dtype="f32", to="f32", tensors=293,
             total=355_000_000, clip=0.1, mix=11),
        # bf16 gradients of a 128-expert layer into fp32 main gradients
        dict(name="clip-experts-bf16", op="clip", dtype="bf16", to="f32", tensors=13,
             total=1_200_000_000, clip=0.01, mix=12),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["ffn", "ffn", "train", "train", "clip"])
    mix = rng.randrange(1 << 30)
    if op == "clip":
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), to=rng.choice(["bf16", "f32"]),
                    tensors=_log(rng, 1, 400), total=_log(rng, 1000, 700_000_000),
                    clip=rng.choice([0.01, 0.3, 2.0]), mix=mix)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    while True:
        if dtype == "f32":
            E, rows = _log(rng, 1, 16), _log(rng, 1, 2048)
            d, f = _log(rng, 32, 768), _log(rng, 64, 2048)
        else:
            E, rows = _log(rng, 1, 128), _log(rng, 1, 16384)
            d, f = _log(rng, 256, 4096, 8), _log(rng, 512, 14336, 8)
        weights = 3 * E * d * f
        if weights <= (1_600_000_000 if op == "train" else 4_000_000_000) and rows * d * f <= 6e11:
            break
    return dict(op=op, dtype=dtype, E=E, rows=rows, d=d, f=f, act=rng.choice(["silu", "gelu"]),
                bias=rng.random() < 0.4, spread=rng.choice(["even", "zipf"]),
                factor=rng.choice([1.25, 2.0]), mix=mix)


def _capacity(case):
    """Rows an expert keeps at most."""
    if case["E"] == 1:
        return case["rows"]
    return max(1, min(case["rows"], math.ceil(case["rows"] / case["E"] * case["factor"])))


def _counts(case):
    """Rows of each expert: the routed demand, cut at the capacity. Goes by the case alone."""
    E, rows = case["E"], case["rows"]
    if E == 1:
        return [rows]
    r = random.Random(case["mix"])
    order = r.sample(range(1, E + 1), E)
    shares = [1.0 if case["spread"] == "even" else k ** -1.2 for k in order]
    ids = r.choices(range(E), weights=shares, k=rows)
    demand = torch.bincount(torch.tensor(ids), minlength=E)
    return demand.clamp(max=_capacity(case)).tolist()


def _sizes(case):
    """Elements of each gradient: large matrices and small vectors, odd sizes among them."""
    r = random.Random(case["mix"])
    n = min(case["tensors"], case["total"])
    raw = [math.exp(r.uniform(-7.0, 0.0)) if r.random() < 0.5 else 1.0 for _ in range(n)]
    scale = case["total"] / sum(raw)
    return [max(1, int(v * scale)) for v in raw]


def _rand(gen, shape, dtype, std):
    return torch.randn(shape, dtype=dtype, device="cuda", generator=gen).mul_(std)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    if case["op"] == "clip":
        grads = [_rand(gen, (n,), dt, 1e-3) for n in _sizes(case)]
        total = sum(g.numel() for g in grads)
        flat = torch.zeros(total, dtype=_DTYPES[case["to"]], device="cuda")
        out = list(flat.split([g.numel() for g in grads]))
        # max_norm as a share of the norm that gradients of this spread have
        return dict(op="clip", grads=grads, flat=flat, out=out,
                    max_norm=case["clip"] * 1e-3 * math.sqrt(total),
                    ws=torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    E, d, f, rows = case["E"], case["d"], case["f"], case["rows"]
    counts = _counts(case)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    s = dict(op=case["op"], act=case["act"], cap=max(counts), offsets=offsets,
             x=_rand(gen, (rows, d), dt, 1.0), y=torch.zeros(rows, d, dtype=dt, device="cuda"),
             h=torch.zeros(rows, f, dtype=dt, device="cuda"))
    for name, shape in (("w_gate", (E, f, d)), ("w_up", (E, f, d)), ("w_down", (E, d, f))):
        s[name] = _rand(gen, shape, dt, 0.02)
    for name, shape in (("b_gate", (E, f)), ("b_up", (E, f)), ("b_down", (E, d))):
        s[name] = _rand(gen, shape, dt, 0.02) if case["bias"] else None
    if case["op"] == "train":
        s["dy"] = _rand(gen, (rows, d), dt, 1.0)
        s["saved"] = torch.zeros(2, rows, f, dtype=dt, device="cuda")
        s["grads"] = {"d" + n: torch.zeros_like(s[n]) for n in
                      ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down") if s[n] is not None}
        s["grads"]["dx_packed"] = torch.zeros_like(s["x"])
    # scratch that a training program keeps: the backward's two hidden gradients and some sums
    scratch = 2 * rows * f * s["x"].element_size() if case["op"] == "train" else 0
    s["ws"] = torch.zeros(scratch + (64 << 20), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _act(z, kind):
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))


def _act_grad(z, kind):
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)


def _to_experts(rows, offsets, cap):
    """[rows, n] -> [E, cap, n] in 32 bits, zero past each expert's rows."""
    at = offsets[:-1, None].long() + torch.arange(cap, device=rows.device)
    inside = at < offsets[1:, None]
    return torch.where(inside[..., None], rows[at.clamp(max=rows.shape[0] - 1)].float(), 0.0)


def _to_rows(padded, offsets, n_rows, dtype):
    """[E, cap, n] -> [rows, n], zero past the last expert's rows."""
    r = torch.arange(n_rows, device=padded.device)
    e = torch.searchsorted(offsets[1:].long(), r, right=True).clamp(max=offsets.numel() - 2)
    at = (r - offsets[e].long()).clamp(0, padded.shape[1] - 1)
    return torch.where((r < offsets[-1])[:, None], padded[e, at], 0.0).to(dtype)


def _linear(a, w, b):
    z = torch.bmm(a, w.float().transpose(1, 2))
    return z if b is None else z + b.float()[:, None]


def _plain_ffn(s):
    x, off, act = s["x"], s["offsets"], s["act"]
    xp = _to_experts(x, off, s["cap"])
    g = _linear(xp, s["w_gate"], s["b_gate"])
    u = _linear(xp, s["w_up"], s["b_up"])
    h = _act(g, act) * u
    y = _to_rows(_linear(h, s["w_down"], s["b_down"]), off, x.shape[0], x.dtype)
    if s["op"] == "ffn":
        return y
    dy = _to_experts(s["dy"], off, s["cap"])
    dh = torch.bmm(dy, s["w_down"].float())
    du = dh * _act(g, act)
    dg = dh * u * _act_grad(g, act)
    dx = torch.bmm(dg, s["w_gate"].float()) + torch.bmm(du, s["w_up"].float())
    out = dict(y=y, dx_packed=_to_rows(dx, off, x.shape[0], x.dtype),
               dw_gate=torch.bmm(dg.transpose(1, 2), xp).to(x.dtype),
               dw_up=torch.bmm(du.transpose(1, 2), xp).to(x.dtype),
               dw_down=torch.bmm(dy.transpose(1, 2), h).to(x.dtype))
    if s["b_gate"] is not None:
        out.update(db_gate=dg.sum(1).to(x.dtype), db_up=du.sum(1).to(x.dtype),
                   db_down=dy.sum(1).to(x.dtype))
    return out


def _plain_clip(s):
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]])
    norm = squares.sum().sqrt()
    factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return norm.float(), torch.cat([(g.float() * factor).to(s["flat"].dtype) for g in s["grads"]])


def run(s):
    if own:
        from mixture_experts_layer_57_b200 import moe
        if s["op"] == "clip":
            norm = moe.moe_clip_grad_norm(s["grads"], s["max_norm"], out=s["out"], ws=s["ws"])
            return norm, s["flat"]
        block = moe.gated_ffn_args(s["x"], s["offsets"], s["w_gate"], s["w_up"], s["w_down"],
                                   b_gate=s["b_gate"], b_up=s["b_up"], b_down=s["b_down"],
                                   act=s["act"], out_dtype=s["y"].dtype, capacity_hint=s["cap"])
        if s["op"] == "ffn":
            moe.moe_gated_ffn(block, y_packed=s["y"], h_packed=s["h"], ws=s["ws"])
            return s["y"]
        moe.moe_gated_ffn(block, y_packed=s["y"], h_packed=s["h"], saved=s["saved"], ws=s["ws"])
        moe.moe_gated_ffn_backward(block, s["dy"], s["h"], s["saved"], s["grads"], ws=s["ws"])
        return dict(y=s["y"], **s["grads"])
    return _plain_clip(s) if s["op"] == "clip" else _plain_ffn(s)


def work(case):
    if case["op"] == "clip":
        n = sum(_sizes(case))
        return dict(bytes=n * (_DTYPES[case["dtype"]].itemsize + _DTYPES[case["to"]].itemsize) + 4,
                    flops=3 * n)
    size, E, d, f = _DTYPES[case["dtype"]].itemsize, case["E"], case["d"], case["f"]
    counts = _counts(case)
    rows, touched = sum(counts), sum(1 for c in counts if c)
    weights = 3 * d * f + ((2 * f + d) if case["bias"] else 0)
    if case["op"] == "ffn":
        return dict(bytes=size * (touched * weights + 2 * rows * d), flops=6 * rows * d * f)
    return dict(bytes=size * (touched * weights + E * weights + 4 * rows * d),
                flops=18 * rows * d * f)


def exact(case, seed):
    """The definition in 64 bits, expert by expert, the gradients by automatic differentiation."""
    s = prepare(case, seed)
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(g.double().pow(2).sum()) for g in s["grads"]))
        factor = min(1.0, s["max_norm"] / (norm + 1e-6))
        return torch.tensor(norm, dtype=torch.float64), torch.cat([g.double() * factor for g in s["grads"]])
    train = case["op"] == "train"
    names = [n for n in ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down") if s[n] is not None]
    out = dict(y=torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda"))
    if train:
        out["dx_packed"] = torch.zeros_like(out["y"])
        out.update({"d" + n: torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in names})
    start = 0
    for e, n in enumerate(_counts(case)):
        if n == 0:
            continue
        rows = slice(start, start + n)
        start += n
        x = s["x"][rows].double().requires_grad_(train)
        p = {k: s[k][e].double().requires_grad_(train) for k in names}
        gate = torch.nn.functional.linear(x, p["w_gate"], p.get("b_gate"))
        gate = torch.nn.functional.silu(gate) if case["act"] == "silu" else torch.nn.functional.gelu(gate)
        up = torch.nn.functional.linear(x, p["w_up"], p.get("b_up"))
        y = torch.nn.functional.linear(gate * up, p["w_down"], p.get("b_down"))
        out["y"][rows] = y.detach()
        if train:
            y.backward(s["dy"][rows].double())
            out["dx_packed"][rows] = x.grad
            for k in names:
                out["d" + k][e] = p[k].grad
        del x, p, gate, up, y
    return out if train else out["y"]
