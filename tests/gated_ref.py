"""The gated expert FFN in 64 bits, forward and backward, with a bound on the error that the
library's arithmetic may have in every element.

The bounds add up, to first order and with 2% for the products of small terms:
  * a sum of n products in fp32: (n + 2) 2^-23 of the sum of the products' magnitudes;
  * a value stored in bf16: 2^-8 of it (half a step), in fp32: 2^-24;
  * the activation and its derivative: 2^-18 of their scale (approximate exponential and division
    in bf16 layers), and what an error of z does to them: |act'| <= 1.13, |act''| <= 0.8.
"""
import math

import torch


def act(z, kind):
    return z * torch.sigmoid(z) if kind == "silu" else 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))


def act_grad(z, kind):
    if kind == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def segment(x, w, kind, dy=None):
    """One expert's rows: x [n, d], w a dict of its parameters (biases may be None), dy [n, d] for
    the gradients. Returns {name: (value, bound before the output's own rounding)}."""
    u = step(x.dtype)
    dd = lambda t: None if t is None else t.double()  # noqa: E731
    xs, wg, wu, wd = x.double(), dd(w["w_gate"]), dd(w["w_up"]), dd(w["w_down"])
    bg, bu, bd = dd(w["b_gate"]), dd(w["b_up"]), dd(w["b_down"])
    n, d = xs.shape
    f = wg.shape[0]
    acc = lambda k: (k + 2) * 2.0 ** -23  # noqa: E731

    def lin(v, m, b, dv=None):
        z = v @ m.T + (0 if b is None else b)
        e = acc(m.shape[1]) * (v.abs() @ m.abs().T + (0 if b is None else b.abs()))
        return z, e if dv is None else e + dv @ m.abs().T

    zg, eg = lin(xs, wg, bg)
    zu, eu = lin(xs, wu, bu)
    a, da = act(zg, kind), act_grad(zg, kind)
    fast = 2.0 ** -18
    ea = 1.13 * eg + fast * (a.abs() + zg.abs() * 2.0 ** -4 + 1e-30)
    eda = 0.8 * eg + fast * (1 + zg.abs())
    h = a * zu
    eh = zu.abs() * ea + a.abs() * eu + u * h.abs()
    y, ey = lin(h, wd, bd, eh)
    out = dict(y=(y, 1.02 * ey))
    if dy is None:
        return out
    q = zu * da
    ea_s = ea + u * a.abs()
    eq_s = zu.abs() * eda + da.abs() * eu + u * q.abs()
    g = dy.double()
    dh = g @ wd
    edh = acc(d) * (g.abs() @ wd.abs())
    du, dg = dh * a, dh * q
    edu = dh.abs() * ea_s + a.abs() * edh + u * du.abs()
    edg = dh.abs() * eq_s + q.abs() * edh + u * dg.abs()
    dx = dg @ wg + du @ wu
    edx = edg @ wg.abs() + edu @ wu.abs() + acc(2 * f) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    out["dx_packed"] = (dx, 1.02 * edx)
    for name, l, el, r, er in (("dw_gate", dg, edg, xs, None), ("dw_up", du, edu, xs, None),
                               ("dw_down", g, None, h, eh)):
        e = acc(n) * (l.abs().T @ r.abs())
        if el is not None:
            e = e + el.T @ r.abs()
        if er is not None:
            e = e + l.abs().T @ er
        out[name] = (l.T @ r, 1.02 * e)
    for name, l, el in (("db_gate", dg, edg), ("db_up", du, edu), ("db_down", g, 0 * g)):
        out[name] = (l.sum(0), 1.02 * (el.sum(0) + acc(n) * l.abs().sum(0)))
    return out


def check(name, got, value, bound):
    """|got - value| within the bound and the rounding to got's type, element by element."""
    tol = bound + step(got.dtype) * (value.abs() + bound) + 1e-37
    err = (got.double() - value).abs()
    worst = float((err / tol).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound at {int((err / tol).argmax())}"
    return worst
