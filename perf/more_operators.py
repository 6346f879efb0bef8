"""The norm in front of a feed-forward block and the block's products in microscaled 8 and 4 bits.

Five operators, in their plain form and through the library, on row-major activations:

  norm        h = x + r,  y = h w / sqrt(mean(h^2) + eps);  y in x's type, or in MX8 blocks
  norm_grad   s = 1 / sqrt(mean(h^2) + eps),  g = dy w,
              dx = dh + s g - h s^3 mean(g h),  dw = sum over rows of dy h s
  quantize    MX blocks of x, from its rows or its columns, and the values that they stand for
  linear      y = act(x W + b) + r,  W in MX4 and x in MX8 or MX4
  gated       h = act(x Wg + bg) (x Wu + bu),  likewise

MX blocks: 32 entries along the contraction share the scale 2^e.  MX8 entries are e4m3 (at most
448), MX4 entries e2m1 (at most 6), to nearest even; e is the smallest for which no entry of the
block rounds beyond the largest value, not under -127.  Rows are stored in whole groups of 256
entries, zeros behind the last one: codes one a byte (MX4: two, the first in the low half) and
scales one a block as e + 127, a weight's rows being its output columns.

`run` takes the plain form (32-bit torch operations, rounded once at the end) where `own` is
false and the library's calls where it is true; `exact` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
EPS = 1e-6
GROUP = 256  # entries that stored rows are filled up to
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def norm_case(name, dtype, M, N, residual, out, pad=0):
    return _named(name, dict(op="norm", dtype=dtype, M=M, N=N, residual=residual, out=out, pad=pad))


def grad_case(name, dtype, M, N, residual, pad=0):
    return _named(name, dict(op="norm_grad", dtype=dtype, M=M, N=N, residual=residual, pad=pad))


def quantize_case(name, dtype, M, K, form, store, pad=0):
    """store: "nk" with the entries of a row side by side, "kn" those of a column."""
    return _named(name, dict(op="quantize", dtype=dtype, M=M, K=K, form=form, store=store, pad=pad))


def product_case(op, name, dtype, M, N, K, x, act, bias=True, residual=False, pad=0):
    """dtype: of bias, residual and output; x: the activations' blocks."""
    return _named(name, dict(op=op, dtype=dtype, M=M, N=N, K=K, x=x, act=act, bias=bias, residual=residual, pad=pad))


def _named(name, c):
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token while answering: the skip connection's sum, normed, as the product's 8-bit operand
        norm_case("norm_token", "bf16", 1, 4096, True, "mx8"),
        # a prompt's or a training step's norm, the sum kept for the layer's next half
        norm_case("norm_4096", "bf16", 4096, 4096, True, "same"),
        # its backward pass, with the gradient that comes down the skip connection
        grad_case("norm_grad_4096", "bf16", 4096, 4096, True),
        # the same in fp32, small and odd, rows with padding between them
        grad_case("norm_grad_odd", "f32", 777, 1025, False, pad=3),
        # a weight stored K x N, laid out in 4 bits once when it is loaded
        quantize_case("quantize_weight", "bf16", 16384, 4096, "mx4", "kn"),
        # a few users' activations in 8 bits, sizes that divide nothing
        quantize_case("quantize_rows33", "f16", 33, 4001, "mx8", "nk", pad=7),
        # one token's output projection: the weights are read once
        product_case("linear", "linear_token", "bf16", 1, 4096, 4096, "mx8", "none", bias=False, residual=True),
        # the down projection of a small serving batch, 4 bits on both sides
        product_case("linear", "linear_rows16", "f16", 16, 4096, 16384, "mx4", "none", residual=True),
        # a prompt's projection with activations in 8 bits, sizes that divide nothing
        product_case("linear", "linear_ragged", "bf16", 4000, 3968, 4001, "mx8", "gelu_tanh", residual=True),
        # the same in 4 bits on both sides
        product_case("linear", "linear_4096", "bf16", 4096, 4096, 4096, "mx4", "gelu_tanh"),
        # a few users' tokens through the gated block
        product_case("gated", "gated_rows33", "bf16", 33, 8190, 4001, "mx8", "silu", bias=False),
        # a prompt's gated block
        product_case("gated", "gated_4096", "bf16", 4096, 8192, 4096, "mx4", "silu", bias=False),
    ]


def draw(rng):
    def size(low, high):
        n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
        return n if rng.random() < 0.4 else max(8, n // 8 * 8)

    op = rng.choice(("norm", "norm_grad", "quantize", "linear", "linear", "gated"))
    dtype, pad = rng.choice(("bf16", "bf16", "f16", "f32")), rng.choice((0, 0, 0, 1, 8))
    while True:
        M, N, K = size(1, 8192), size(64, 16384), size(128, 16384)
        if rng.random() < 0.35:
            M = rng.randint(1, 48)  # single tokens and small batches
        if op in ("norm", "norm_grad") and M * N <= 1 << 26 or op == "quantize" and N * K <= 1 << 26:
            break
        if op in ("linear", "gated") and N >= 128 and M * N * K * (2 if op == "gated" else 1) <= 2.7e11:
            break
    if op == "norm":
        return norm_case(None, dtype, M, N, rng.random() < 0.7, rng.choice(("same", "mx8")), pad)
    if op == "norm_grad":
        return grad_case(None, dtype, M, N, rng.random() < 0.6, pad)
    if op == "quantize":
        return quantize_case(None, dtype, N, K, rng.choice(("mx4", "mx8")), rng.choice(("nk", "kn")), pad)
    act = rng.choice(ACTS if op == "linear" else ("silu", "gelu", "gelu_tanh", "relu"))
    return product_case(op, None, dtype, M, N, K, rng.choice(("mx8", "mx4")), act, bias=rng.random() < 0.5,
                        residual=op == "linear" and rng.random() < 0.5, pad=pad)


def _filled(K):
    return -(-K // GROUP) * GROUP


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t, M, pad = TYPES[case["dtype"]], case["M"], case["pad"]

    def rows(r, c, scale=1.0):
        """r x c values, `pad` elements apart."""
        return torch.randn(r, c + pad, generator=gen, device="cuda").mul_(scale).to(t)[:, :c]

    def empty(r, c):
        return torch.empty(r, c + pad, dtype=t, device="cuda")[:, :c]

    def stored(r, K, form):
        """Codes and scales of an r x K matrix to be written."""
        width = _filled(K)
        return (torch.empty(r, width if form == "mx8" else width // 2, dtype=torch.uint8, device="cuda"),
                torch.empty(r, width // 32, dtype=torch.uint8, device="cuda"))

    def gain(n):
        return (1 + 0.2 * torch.randn(n, generator=gen, device="cuda")).to(t)

    s = dict(case=case)
    if case["op"] == "norm":
        N = case["N"]
        s.update(X=rows(M, N), w=gain(N), R=None, H=None, mx=None, Y=None, V=None)
        if case["residual"]:
            s.update(R=rows(M, N, 2.0), H=empty(M, N))
        if case["out"] == "mx8":
            s.update(mx=stored(M, N, "mx8"), V=torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
        else:
            s.update(Y=empty(M, N))
    elif case["op"] == "norm_grad":
        N = case["N"]
        s.update(H=rows(M, N, 2.0), dY=rows(M, N), w=gain(N), dH=rows(M, N) if case["residual"] else None,
                 dX=empty(M, N), dw=torch.empty(N, dtype=t, device="cuda"))
    elif case["op"] == "quantize":
        K = case["K"]
        s.update(X=rows(M, K, K ** -0.5) if case["store"] == "nk" else rows(K, M, K ** -0.5).t(),
                 mx=stored(M, K, case["form"]), V=torch.empty(M, K, dtype=torch.bfloat16, device="cuda"))
    else:
        N, K = case["N"], case["K"]

        def blocks(r, form, scale):
            """Codes and scales of r rows of K normal values."""
            x = torch.randn(r, K, generator=gen, device="cuda").mul_(scale)
            return _store(*_entries(x, form), form)

        s.update(X=blocks(M, case["x"], 1.0), Y=empty(M, N), R=rows(M, N) if case["residual"] else None)
        for i in ("g", "u") if case["op"] == "gated" else ("",):
            s["W" + i] = blocks(N, "mx4", K ** -0.5)
            s["b" + i] = torch.randn(N, generator=gen, device="cuda").mul_(0.5).to(t) if case["bias"] else None
    return s


# ---- the plain form ------------------------------------------------------------------------


def _entries(x, form):
    """The entries (values of e4m3 or e2m1) of fp32 rows in whole groups, and the scales' bytes."""
    M, K = x.shape
    whole = torch.zeros(M, _filled(K), device=x.device)
    whole[:, :K] = x
    b = whole.view(M, -1, 32)
    # the scale from the bits of the largest entry: one more where it would round beyond the largest value
    up, down = (0x17FFFF, 8) if form == "mx8" else (0x200000, 2)
    e = (((b.abs().amax(-1).view(torch.int32) + up) >> 23) - down).clamp_min(0)
    a = b * ((254 - e) << 23).view(torch.float32)[..., None]
    # steps of the entries' own binade, from the exponent of each, not under that of the smallest normal
    low, bits = (-6, 3) if form == "mx8" else (0, 1)
    step = (((a.view(torch.int32) >> 23) & 255) - 127).clamp_min(low) - bits
    q = torch.round(a * ((127 - step) << 23).view(torch.float32)) * ((127 + step) << 23).view(torch.float32)
    return q, e


def _store(q, e, form):
    """Bytes of entries and scales."""
    if form == "mx8":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        n = torch.bucketize(q.abs(), torch.tensor(E2M1, device=q.device)) + 8 * torch.signbit(q)
        codes = (n[..., 0::2] | n[..., 1::2] << 4).to(torch.uint8)
    return codes.reshape(q.shape[0], -1), e.to(torch.uint8)


def _values(q, e):
    """What entries and scales' bytes stand for, in fp32."""
    s = torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)
    return (q * s[..., None]).flatten(1)


def _decoded(stored, form):
    codes, e = stored
    if form == "mx8":
        q = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        n = codes.int()
        q = table[torch.stack((n & 15, n >> 4), -1).flatten(1)]
    return _values(q.view(q.shape[0], -1, 32), e.int())


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain(s):
    c = s["case"]
    t = TYPES[c["dtype"]]
    if c["op"] == "norm":
        h = s["X"].float()
        if s["R"] is not None:
            h = h + s["R"].float()
        y = h * (1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)) * s["w"].float()
        out = {"H": h.to(t)} if s["R"] is not None else {}
        if c["out"] == "mx8":
            return dict(out, values=_values(*_entries(y, "mx8"))[:, :c["N"]].to(torch.bfloat16))
        return dict(out, Y=y.to(t))
    if c["op"] == "norm_grad":
        h, dy = s["H"].float(), s["dY"].float()
        r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
        g = dy * s["w"].float()
        dx = r * g - h * (r * r * r * (g * h).mean(1, keepdim=True))
        if s["dH"] is not None:
            dx = dx + s["dH"].float()
        return {"dX": dx.to(t), "dw": (dy * h * r).sum(0).to(t)}
    if c["op"] == "quantize":
        return {"values": _values(*_entries(s["X"].float(), c["form"]))[:, :c["K"]].to(torch.bfloat16)}
    x = _decoded(s["X"], c["x"])

    def project(w, b):
        z = x @ _decoded(s[w], "mx4").t()
        return z if s[b] is None else z + s[b].float()

    if c["op"] == "gated":
        return {"H": (_act(project("Wg", "bg"), c["act"]) * project("Wu", "bu")).to(t)}
    y = _act(project("W", "b"), c["act"])
    return {"Y": (y if s["R"] is None else y + s["R"].float()).to(t)}


# ---- the library's calls -------------------------------------------------------------------


def _own(s):
    from software_pipelined_tiled_loop_amd import binding as pg
    c = s["case"]
    if c["op"] == "norm":
        pg.rms_norm(s["X"], s["w"], s["Y"], residual=s["R"], H=s["H"], mx=s["mx"], eps=EPS)
        out = {"H": s["H"]} if s["R"] is not None else {}
        if c["out"] == "mx8":
            return dict(out, values=pg.mx_dequantize(s["mx"], s["V"]))
        return dict(out, Y=s["Y"])
    if c["op"] == "norm_grad":
        pg.rms_norm_backward(s["dY"], s["H"], s["w"], dH=s["dH"], dX=s["dX"], dweight=s["dw"], eps=EPS)
        return {"dX": s["dX"], "dw": s["dw"]}
    if c["op"] == "quantize":
        return {"values": pg.mx_dequantize(pg.mx_quantize(s["X"], s["mx"]), s["V"])}
    if c["op"] == "gated":
        return {"H": pg.mx_gated(s["X"], s["Wg"], s["Wu"], s["Y"], bias_g=s["bg"], bias_u=s["bu"], act=c["act"])}
    return {"Y": pg.mx_linear(s["X"], s["W"], s["Y"], bias=s["b"], residual=s["R"], act=c["act"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without, and its exact values -------------------------------------


def work(case):
    M, e = case["M"], BYTES[case["dtype"]]
    if case["op"] == "norm":
        N, r = case["N"], case["residual"]
        return {"bytes": M * N * (e * (1 + 2 * r) + (2 if case["out"] == "mx8" else e)) + N * e, "flops": 5 * M * N}
    if case["op"] == "norm_grad":
        N = case["N"]
        return {"bytes": M * N * e * (3 + case["residual"]) + 2 * N * e, "flops": 10 * M * N}
    K = case["K"]
    if case["op"] == "quantize":
        return {"bytes": M * K * (e + 2), "flops": 4 * M * K}
    N, W = case["N"], 2 if case["op"] == "gated" else 1
    x, w = (1 if case["x"] == "mx8" else 0.5) + 1 / 32, 0.5 + 1 / 32
    return {"bytes": M * K * x + W * N * (K * w + e * case["bias"]) + e * M * N * (1 + case["residual"]),
            "flops": 2 * W * M * N * K}


def _times(x, e):
    """x 2^e, exactly."""
    return x * ((e.long() + 1023) << 52).view(torch.float64)


def _exact_blocks(x, form):
    """The values of a matrix's blocks, in 64 bits, by comparison with every value of the format."""
    M, K = x.shape
    grid = [v * 1.0 for v in E2M1] if form == "mx4" else [
        m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:-1]
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    over = 464.0 if form == "mx8" else 7.0  # half way to the value behind the largest: that one is even in MX4, odd in MX8
    whole = x.new_zeros(M, _filled(K))
    whole[:, :K] = x
    b = whole.view(M, -1, 32)
    most = b.abs().amax(-1)
    e = torch.frexp(most / over)[1].clamp_min(-127)  # over 2^e > most
    for _ in range(2):
        small = _times(most, 1 - e)
        fits = (small <= over if form == "mx8" else small < over) & (e > -127)
        e = torch.where(fits, e - 1, e)
    a = _times(b.abs(), -e[..., None])
    at = torch.searchsorted(grid, a.contiguous()).clamp(1, grid.numel() - 1)
    lo, hi = grid[at - 1], grid[at]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (at % 2 == 0))
    v = _times(torch.where(up, hi, lo), e[..., None]).copysign(b)
    return v.flatten(1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def wide(v):
        return None if v is None else v.double()

    def table(form):
        if form == "mx4":
            half = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
            return torch.cat((half, -half))
        n = torch.arange(256, device="cuda")
        m, e = (n & 7).double(), n >> 3 & 15
        v = torch.where(e > 0, _times(8 + m, e - 10), m * 2.0 ** -9)
        return torch.where(n < 128, v, -v)

    def matrix(stored, form):
        codes, scales = stored[0].long(), stored[1].long()
        if form == "mx4":
            codes = torch.stack((codes % 16, codes // 16), 2).reshape(codes.shape[0], -1)
        return _times(table(form)[codes], (scales - 127).repeat_interleave(32, 1))

    if op == "norm":
        h = wide(s["X"]) if s["R"] is None else wide(s["X"]) + wide(s["R"])
        y = h / (h.square().sum(1) / h.shape[1] + EPS).sqrt()[:, None] * wide(s["w"])
        out = {} if s["R"] is None else {"H": h}
        return dict(out, values=_exact_blocks(y, "mx8")) if case["out"] == "mx8" else dict(out, Y=y)
    if op == "norm_grad":
        h, w = wide(s["H"]).requires_grad_(), wide(s["w"]).requires_grad_()
        y = h * (h.square().sum(1) / h.shape[1] + EPS).rsqrt()[:, None] * w
        dx, dw = torch.autograd.grad(y, (h, w), wide(s["dY"]))
        return {"dX": dx if s["dH"] is None else dx + wide(s["dH"]), "dw": dw}
    if op == "quantize":
        return {"values": _exact_blocks(wide(s["X"]), case["form"])}
    x, name = matrix(s["X"], case["x"]), case["act"]

    def f(z):
        if name == "none":
            return z
        if name == "relu":
            return z.clamp_min(0)
        if name == "silu":
            return z * torch.special.expit(z)
        if name == "gelu":
            return z * torch.special.ndtr(z)
        # (1 + tanh a) / 2 is the logistic function of 2a
        return z * torch.special.expit(math.sqrt(8 / math.pi) * z * (1 + 0.044715 * z.square()))

    def product(w, b):
        z = torch.mm(x, matrix(s[w], "mx4").t())
        return z if s[b] is None else z + wide(s[b])

    if op == "gated":
        return {"H": f(product("Wg", "bg")) * product("Wu", "bu")}
    y = f(product("W", "b"))
    return {"Y": y if s["R"] is None else y + wide(s["R"])}
