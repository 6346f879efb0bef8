"""Plain 64-bit forms of the norm and of the microscaled operators, and bounds on their rounding.

s = 2^-24 is half a step of fp32.

* norm: h = x + r rounds once (s |h|).  Its squares are summed along chains: eight a group of
  columns and thread, at most N / 8192 + 4 groups long, then at most 6 + 16 sums of waves: a sum of
  positive terms whose longest chain has c links is off by at most c s of itself, here c = 64 + N / 1024.
  With 3 s for each square (two from h) and s for the mean and the sum with eps, s the square root's and the
  quotient's roundings, 1 / sqrt(.) is off by (c + 5) / 2 s + 3 s of itself, and y, three products on, by
  (c / 2 + 10) s |y| and s |h| of h moved through: in all (c / 2 + 12) s |y|.
* norm backward: rs as above, relative error er = (c / 2 + 6) s (h is given).  sum(g h) is off by at most
  (c + 3) s sum|g h|.  dx = dh + rs g - h rs^2 m', m' = rs mean(g h): each term's factors' errors and roundings,
  at most rs |g| (er + 4 s) + |h| rs^3 ((3 er + 8 s) |mean| + (c + 4) s mean|g h|) + 2 s (|terms|).
  dw: each term rs |dy h| (er + 3 s), and its sum over M rows (M + 8) s.
* MX outputs of a y that is off by e hold, at their own scale, what rounding some value of [y - e, y + e] gives
  (rounding is monotone), and their scale is that of some largest entry of [amax - e, amax + e].
* products: entries, scales and their products are exact.  Sums over n stored entries in fp32, in any order, are
  off by (n + 8) s sum|a b|.  Of e4m3 operands the matrix cores add, for 16-bit outputs, eight neighbouring products
  aligned to the largest and keep 13 bits below its leading one: seven of them lose less than 2^-13 of the largest each.
  Products far below that may vanish; none is below 2^-149 here.
"""
import torch

from linear_reference import S, act_bound, half_step, round_out, tiny  # noqa: F401

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E4M3 = tuple(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8))[:-1]


def filled(K):
    return -(-K // 256) * 256


def scale_of(most, form):
    """The smallest e from -127 on for which an entry of size `most` does not round beyond the largest value."""
    def fits(e):
        a = torch.ldexp(most, -e)
        return a <= 464 if form == "mx8" else a < 7
    e = torch.where(most > 0, torch.frexp(most)[1] - (8 if form == "mx8" else 2), torch.full_like(most, -127).int())
    e = e.clamp_min(-127)
    for _ in range(4):
        e = torch.where(fits(e), e, e + 1)
    for _ in range(4):
        e = torch.where(fits(e - 1) & (e > -127), e - 1, e)
    assert bool((fits(e) | (most == 0)).all())
    return e


def nearest(a, form):
    """a >= 0 rounded to the format's values, ties to even codes, largest value beyond it."""
    grid = torch.tensor(E4M3 if form == "mx8" else E2M1, dtype=torch.float64)
    at = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
    lo, hi = grid[at - 1], grid[at]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (at % 2 == 0))
    return torch.where(up, hi, lo)


def blocks(x):
    """rows x K as rows x blocks x 32, filled up."""
    w = x.new_zeros(x.shape[0], filled(x.shape[1]))
    w[:, :x.shape[1]] = x
    return w.view(x.shape[0], w.shape[1] // 32, 32)


def quantize(x, form):
    """(bytes of codes, bytes of scales) of a matrix of finite or other values."""
    b = blocks(x.double().cpu())
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    e = scale_of(b.abs().amax(-1), form)
    q = nearest(torch.ldexp(b.abs(), -e[..., None]), form)
    grid = torch.tensor(E4M3 if form == "mx8" else E2M1, dtype=torch.float64)
    code = torch.searchsorted(grid, q.contiguous()).int()
    code = code + (128 if form == "mx8" else 8) * (torch.signbit(b) & ~bad[..., None]).int()
    code = code.flatten(1)
    if form == "mx4":
        code = code[:, 0::2] | code[:, 1::2] << 4
    s = torch.where(bad, torch.full_like(e, 255), e + 127)
    return code.to(torch.uint8), s.to(torch.uint8)


def entries(Q, form):
    Q = Q.cpu().view(torch.uint8).long()
    if form == "mx4":
        t = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64)
        return t[torch.stack((Q & 15, Q >> 4), -1).flatten(1)]
    t = torch.tensor(E4M3 + (float("nan"),), dtype=torch.float64)
    return torch.cat((t, -t))[Q]


def values(Q, S_, form):
    """What blocks stand for, all stored entries."""
    s = S_.cpu().view(torch.uint8).int()
    scale = torch.where(s == 255, torch.full(s.shape, float("nan"), dtype=torch.float64),
                        torch.ldexp(torch.ones(s.shape, dtype=torch.float64), s - 127))
    return entries(Q, form) * scale.repeat_interleave(32, 1)


def form_of(mx):
    return "mx8" if mx[0].shape[1] == 32 * mx[1].shape[1] else "mx4"


def chain(N):
    return 64 + N / 1024


def norm(x, r, w, eps):
    """(h, its error), (y, its error), not yet rounded."""
    h = x.double().cpu() if r is None else x.double().cpu() + r.double().cpu()
    rs = 1 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    y = h * rs if w is None else h * rs * w.double().cpu()
    return (h, S * h.abs() * (r is not None)), (y, (chain(h.shape[1]) / 2 + 12) * S * y.abs())


def norm_backward(dy, h, w, dh, eps):
    dy, h = dy.double().cpu(), h.double().cpu()
    N, M = h.shape[1], h.shape[0]
    c = chain(N)
    er = (c / 2 + 6) * S
    rs = 1 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    g = dy if w is None else dy * w.double().cpu()
    mean, mag = (g * h).mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    a, b = rs * g, h * rs ** 3 * mean
    dx = a - b if dh is None else dh.double().cpu() + a - b
    edx = a.abs() * (er + 4 * S) + h.abs() * rs ** 3 * ((3 * er + 8 * S) * mean.abs() + (c + 4) * S * mag)
    edx = edx + 2 * S * (a.abs() + b.abs() + dx.abs())
    t = dy * h * rs
    return (dx, edx), (t.sum(0), t.abs().sum(0) * (er + 3 * S + (M + 8) * S))


def check_blocks(mx, y, e, what):
    """MX blocks of a y that is off by at most e."""
    form = form_of(mx)
    Q, s = mx[0].cpu(), mx[1].cpu().view(torch.uint8).int()
    b, eb = blocks(y), blocks(e)
    k = s - 127
    most, slack = b.abs().amax(-1), eb.amax(-1)
    lo, hi = scale_of((most - slack).clamp_min(0), form), scale_of(most + slack, form)
    assert bool(((k >= lo) & (k <= hi)).all()), "%s: scales" % what
    v = entries(Q, form).view(b.shape)
    signed = lambda t: nearest(torch.ldexp(t.abs(), -k[..., None]), form).copysign(t)  # noqa: E731
    low, high = signed(b - eb), signed(b + eb)
    bad = ~((v >= low) & (v <= high))
    assert not bool(bad.any()), "%s: %d codes, the first at %s" % (what, int(bad.sum()), bad.nonzero()[0].tolist())


def product(x, w, xform, dtype):
    """X W^T of values of stored entries, and how far the sums may be off."""
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    e = (x.shape[1] + 8) * S * mag
    if xform == "mx8" and dtype != torch.float32 and x.shape[1]:
        most = lambda t: t.abs().view(t.shape[0], t.shape[1] // 8, 8).amax(-1)  # noqa: E731
        e = e + 7 * 2.0 ** -13 * (most(x) @ most(w).t())
    return z, e


def linear(X, W, b, R, act, dtype):
    x = values(*X, form_of(X))
    z, ez = product(x, values(*W, "mx4"), form_of(X), dtype)
    if b is not None:
        z = z + b.double().cpu()
        ez = ez + 2 * S * (z.abs() + b.double().cpu().abs())
    v, ev = act_bound(z, ez, act)
    if R is not None:
        v = v + R.double().cpu()
        ev = ev + S * (v.abs() + ev)
    return round_out(v, ev, dtype)


def gated(X, Wg, Wu, bg, bu, act, dtype):
    x, f = values(*X, form_of(X)), form_of(X)
    g, eg = product(x, values(*Wg, "mx4"), f, dtype)
    u, eu = product(x, values(*Wu, "mx4"), f, dtype)
    if bg is not None:
        g, eg = g + bg.double().cpu(), eg + 2 * S * (g.abs() + bg.double().cpu().abs())
    if bu is not None:
        u, eu = u + bu.double().cpu(), eu + 2 * S * (u.abs() + bu.double().cpu().abs())
    v, ev = act_bound(g, eg, act)
    h = v * u
    return round_out(h, ev * u.abs() + v.abs() * eu + ev * eu + S * h.abs(), dtype)


def close(got, want, what):
    v, e = want
    d = (got.double().cpu() - v).abs()
    bad = ~(d <= e)
    assert not bool(bad.any()), "%s: %d of %d off, the worst by %.3g of its bound at %s" % (
        what, int(bad.sum()), d.numel(), float((d / e.clamp_min(1e-300)).nan_to_num(float("inf")).max()),
        bad.nonzero()[0].tolist())
