"""Plain 64-bit forms of the feed-forward operators, and bounds on their rounding.

Each function returns (value, bound): the exact value in float64 and how far a
correct result may be from it, element by element.  u is half a step of a
type relative to the value (finfo.eps / 2); s = 2^-24 that of fp32.

* A sum of n products in fp32, in any order, is off by at most about
  n s sum|a b| (each of the n additions rounds once, and the products inside
  the matrix cores at most once): (n + 8) s sum|a b| covers the few
  additions of bias and of split sums too.
* act is evaluated on a z that is off by dz: |act'| <= 1.13 for every
  activation here, so it moves by at most 1.13 dz.  The evaluation itself
  rounds an exponent argument |a| <= 120 before exp2 (a s relative to e), and
  exp2, 1 + e, 1 / (1 + e) and the last product once or twice each: with
  e / (1 + e)^2 |a| <= 0.23 the value is off by at most 8 s (|z| + |act|),
  and gelu's fit by 7e-8 < 2 s more.
* act' is bounded by 1.13 and moves by at most |act''| <= 1 times dz (no dz
  here: Z is an input); its evaluation has the same roundings on factors up to
  |z| p (1 - p) P <= 1.3: 32 s (1 + |z| min(1, ..)) is used, 32 s (1 + min(|z|, 8)).
* dZ is rounded to the operand type before the products (u |dZ|) unless act is
  none; sums of gradients for the biases are not.
* The output rounds once: u_out |value|.  Values below the type's smallest
  normal are off by at most half its smallest subnormal step instead.
"""
import math

import torch

S = 2.0 ** -24
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    f = torch.finfo(dtype)
    return f.tiny * f.eps


def act64(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        p = torch.special.expit(z)
        return p + z * p * torch.special.expit(-z)
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


WHERE = "cpu"  # the large cases set it to the GPU for their time


def d(t):
    return None if t is None else t.detach().to(WHERE).double()


def round_out(v, e, dtype):
    return v, e + half_step(dtype) * (v.abs() + e) + tiny(dtype)


def project(X, W, b):
    x, w = d(X), d(W)
    z, n = x @ w, X.shape[1]
    mag = x.abs() @ w.abs()
    if b is not None:
        z, mag = z + d(b), mag + d(b).abs()
    return z, (n + 8) * S * mag


def act_bound(z, ez, act):
    v = act64(z, act)
    if act == "none":
        return v, ez
    return v, 1.13 * ez + 10 * S * (z.abs() + v.abs())


def linear(X, W, b, R, act, y_dtype):
    z, ez = project(X, W, b)
    v, ev = act_bound(z, ez, act)
    if R is not None:
        v = v + d(R)
        ev = ev + S * (v.abs() + ev)
    return round_out(v, ev, y_dtype), round_out(z, ez, X.dtype)


def gated(X, Wg, Wu, bg, bu, act, h_dtype):
    g, eg = project(X, Wg, bg)
    u, eu = project(X, Wu, bu)
    v, ev = act_bound(g, eg, act)
    h = v * u
    eh = ev * u.abs() + v.abs() * eu + ev * eu + S * h.abs()
    return round_out(h, eh, h_dtype), round_out(g, eg, X.dtype), round_out(u, eu, X.dtype)


def slope_bound(z, act):
    s = slope64(z, act)
    if act in ("none", "relu"):
        return s, torch.zeros_like(s)
    return s, 32 * S * (1 + z.abs().clamp_max(8))


def products(parts, X, dtype, g_dtype, rounded):
    """parts: (dZ, its error, W) of each plane -> dX, and (dW, db) of each plane."""
    x = d(X)
    u = half_step(dtype) if rounded else 0.0
    t = tiny(dtype) if rounded else 0.0
    dx, edx, outs = 0, 0, []
    for dz, e, W in parts:
        w = d(W)
        er = e + u * (dz.abs() + e) + t          # of the operand of the products
        mag = dz.abs() + er
        dx = dx + dz @ w.t()
        edx = edx + er @ w.abs().t() + (len(parts) * dz.shape[1] + 8) * S * (mag @ w.abs().t())
        dw = x.t() @ dz
        edw = x.abs().t() @ er + (dz.shape[0] + 8) * S * (x.abs().t() @ mag)
        db = dz.sum(0)
        edb = e.sum(0) + (dz.shape[0] + 8) * S * (dz.abs() + e).sum(0)
        outs.append((round_out(dw, edw, g_dtype), round_out(db, edb, g_dtype)))
    return round_out(dx, edx, dtype), outs


def linear_backward(dY, X, W, Z, act, g_dtype):
    dy = d(dY)
    if act == "none":
        dz, e = dy, torch.zeros_like(dy)
    else:
        s, es = slope_bound(d(Z), act)
        dz = dy * s
        e = dy.abs() * es + S * dz.abs()
    dx, ((dw, db),) = products([(dz, e, W)], X, X.dtype, g_dtype, act != "none")
    return dx, dw, db


def gated_backward(dH, X, Wg, Wu, G, U, act, g_dtype):
    dh, g, u = d(dH), d(G), d(U)
    s, es = slope_bound(g, act)
    v, ev = act_bound(g, torch.zeros_like(g), act)
    dg, du = dh * u * s, dh * v
    eg = (dh * u).abs() * es + 2 * S * dg.abs()
    eu = dh.abs() * ev + S * du.abs()
    dx, ((dwg, dbg), (dwu, dbu)) = products([(dg, eg, Wg), (du, eu, Wu)], X, X.dtype, g_dtype, True)
    return dx, dwg, dwu, dbg, dbu


def check(name, got, want):
    value, bound = want
    got = d(got)
    bad = ~((got - value).abs() <= bound)
    if bool(bad.any()):
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError("%s%s = %r, exact %r, bound %.3g (%d of %d off)" % (
            name, at, float(got[at]), float(value[at]), float(bound[at]), int(bad.sum()), bad.numel()))
