"""The backward passes over the whole range of fp16 gradients.

dG = dH U act'(G) and dU = dH act(G) of fp16 tensors lie between 2^-48 and 2^33
and beyond, fp16 itself between 2^-24 and 2^16.  The operators hold them scaled by a
power of two for each row (in dX) and each column (in dW), so what the formula
keeps finite stays finite and what it keeps different from zero does not vanish
while its row or column has nothing 2^29 times larger.

Bounds.  A scaled value has its row's (column's) largest entry in [2^14, 2^15):
rounding it to fp16 is off by u |dZ|, u = 2^-11, or by half of fp16's smallest step
2^-24, which in units of that largest entry m is at most 2^-25 m / 2^14 = 2^-39 m.
Everything else is as in linear_reference.py.  Rows are scaled by the largest
entry of dG and dU together, as both add up in dX.
"""
import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
F16 = torch.float16
S = ref.S
FLOOR = 2.0 ** -39


@pytest.fixture(scope="module")
def pg():
    from software_pipelined_tiled_loop_amd import binding
    return binding


def say(*a):
    print("[case]", *a, flush=True)


def products(parts, X, g_dtype, rounded=True):
    """parts: (dZ, its error, W) of each plane -> dX, [(dW, db)] with their bounds, fp16 operands."""
    x, u = ref.d(X), ref.half_step(F16) if rounded else 0.0
    row = torch.stack([(dz.abs() + e).amax(1) for dz, e, _ in parts]).amax(0)
    dx, edx, outs = 0, 0, []
    for dz, e, W in parts:
        w = ref.d(W)
        er = e + u * (dz.abs() + e)
        floor_r = FLOOR * row[:, None] if rounded else 0.0
        floor_c = FLOOR * (dz.abs() + e).amax(0)[None, :] if rounded else 0.0
        mag = dz.abs() + er + floor_r
        dx = dx + dz @ w.t()
        edx = edx + (er + floor_r) @ w.abs().t() + (len(parts) * dz.shape[1] + 8) * S * (mag @ w.abs().t())
        mag = dz.abs() + er + floor_c
        dw = x.t() @ dz
        edw = x.abs().t() @ (er + floor_c) + (dz.shape[0] + 8) * S * (x.abs().t() @ mag)
        db = dz.sum(0)
        edb = e.sum(0) + (dz.shape[0] + 8) * S * (dz.abs() + e).sum(0)
        outs.append((ref.round_out(dw, edw, g_dtype), ref.round_out(db, edb, g_dtype)))
    return ref.round_out(dx, edx, F16), outs


def gated_parts(dH, G, U, act, Wg, Wu):
    dh, g, u = ref.d(dH), ref.d(G), ref.d(U)
    s, es = ref.slope_bound(g, act)
    v, ev = ref.act_bound(g, torch.zeros_like(g), act)
    dg, du = dh * u * s, dh * v
    return [(dg, (dh * u).abs() * es + 2 * S * dg.abs(), Wg), (du, dh.abs() * ev + S * du.abs(), Wu)]


def linear_part(dY, Z, act, W):
    dy = ref.d(dY)
    s, es = ref.slope_bound(ref.d(Z), act)
    return [(dy * s, dy.abs() * es + S * (dy * s).abs(), W)]


def randn(gen, *shape):
    return torch.randn(*shape, generator=gen)


def signs(gen, *shape):
    return torch.randint(0, 2, shape, generator=gen).float() * 2 - 1


def gpu16(t):
    return t.to(F16).cuda()


def run_gated(pg, dH, X, Wg, Wu, G, U, act, g_dtype, order, bias=True):
    M, N, K = dH.shape[0], dH.shape[1], X.shape[1]

    def weight_out():
        return torch.full((K, N), 7.0, dtype=g_dtype, device="cuda") if order == "kn" else torch.full(
            (N, K), 7.0, dtype=g_dtype, device="cuda").t()

    out = dict(dX=torch.full((M, K), 7.0, dtype=F16, device="cuda"), dWg=weight_out(), dWu=weight_out())
    if bias:
        out.update(dbias_g=torch.empty(N, dtype=g_dtype, device="cuda"), dbias_u=torch.empty(N, dtype=g_dtype, device="cuda"))
    pg.gated_backward(dH, X, Wg, Wu, G, U, act=act, **out)
    torch.cuda.synchronize()
    return out


def check_gated(pg, dH, X, Wg, Wu, G, U, act, g_dtype, order, bias=True):
    got = run_gated(pg, dH, X, Wg, Wu, G, U, act, g_dtype, order, bias)
    dx, ((dwg, dbg), (dwu, dbu)) = products(gated_parts(dH, G, U, act, Wg, Wu), X, g_dtype)
    want = dict(dX=dx, dWg=dwg, dWu=dwu, dbias_g=dbg, dbias_u=dbu)
    assert all(bool(torch.isfinite(t).all()) for t in got.values())
    for k, v in got.items():
        ref.check(k, v, want[k])
    return got, want


SIZES = [(1, 40, 24), (70, 130, 65), (300, 264, 136), (1000, 333, 129)]


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gated_gradients_beyond_the_largest_fp16(pg, M, N, K, order):
    """dH = U = 300: |dG| up to 1e5, finite fp32 weight gradients, and dX finite through small weights."""
    gen = torch.Generator().manual_seed(M)
    say("large", (M, N, K), order)
    dH, U = gpu16(300 * signs(gen, M, N)), gpu16(300 * signs(gen, M, N))
    G, X = gpu16(randn(gen, M, N) + 1), gpu16(randn(gen, M, K))
    Wg, Wu = (gpu16(randn(gen, K, N) * 2.0 ** -10) for _ in range(2))
    check_gated(pg, dH, X, Wg, Wu, G, U, "silu", torch.float32, order)


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gated_gradients_below_the_smallest_fp16(pg, M, N, K, order):
    """dH about 1e-6, U about 1e-2: dG about 1e-8, in fp32 weight gradients and, through weights of 200, in dX."""
    gen = torch.Generator().manual_seed(M + 1)
    say("small", (M, N, K), order)
    dH, U = gpu16(1e-6 * (1 + randn(gen, M, N).abs()) * signs(gen, M, N)), gpu16(1e-2 * randn(gen, M, N))
    G, X = gpu16(1e-2 * randn(gen, M, N)), gpu16(randn(gen, M, K))
    Wg, Wu = (gpu16(randn(gen, K, N) * 200) for _ in range(2))
    got, _ = check_gated(pg, dH, X, Wg, Wu, G, U, "gelu", torch.float32, order)
    assert bool((got["dWg"] != 0).any()) and bool((got["dWu"] != 0).any())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu", "none"])
@pytest.mark.parametrize("order", ["kn", "nk"])
def test_gated_rows_and_columns_of_their_own_size(pg, act, order):
    """Rows of dH over 2^30 and columns of U over 2^12: each row of dX and column of dW keeps its own accuracy."""
    M, N, K = 260, 200, 72
    say("mixed", act, order)
    gen = torch.Generator().manual_seed(3)
    rows = 2.0 ** (torch.arange(M) % 31 - 19).float()
    cols = 2.0 ** (torch.arange(N) % 13 - 9).float()
    dH = gpu16(rows[:, None] * (1 + 0.5 * torch.rand(M, N, generator=gen)) * signs(gen, M, N))
    U = gpu16(cols * randn(gen, M, N))
    G, X = gpu16(0.5 + 0.25 * randn(gen, M, N).clamp(-1, 1)), gpu16(randn(gen, M, K))
    Wg, Wu = (gpu16(randn(gen, K, N) * 2.0 ** -3) for _ in range(2))
    check_gated(pg, dH, X, Wg, Wu, G, U, act, torch.float32, order)


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("scale", [2.0 ** 15, 2.0 ** -20])
def test_linear_gradients_at_both_ends(pg, scale, order):
    M, N, K = 190, 270, 88
    say("linear", scale, order)
    gen = torch.Generator().manual_seed(9)
    dY = gpu16(scale * (1 + 0.9 * torch.rand(M, N, generator=gen)) * signs(gen, M, N))
    # slopes from 1.13 (dY act' passes 65504) down to 1e-4
    Z, X = gpu16(1.4 + 0.1 * randn(gen, M, N) if scale > 1 else -3 + randn(gen, M, N).clamp(-2, 2)), gpu16(randn(gen, M, K))
    W = gpu16(randn(gen, K, N) * (2.0 ** -9 if scale > 1 else 2.0 ** 5))
    W = W if order == "kn" else W.t().contiguous().t()
    dW = torch.empty(K, N, device="cuda") if order == "kn" else torch.empty(N, K, device="cuda").t()
    dX, db = torch.empty(M, K, dtype=F16, device="cuda"), torch.empty(N, device="cuda")
    for act in ("gelu", "silu"):
        pg.linear_backward(dY, X, W, Z=Z, act=act, dX=dX, dW=dW, dbias=db)
        torch.cuda.synchronize()
        dx, ((dw, dbias),) = products(linear_part(dY, Z, act, W), X, torch.float32)
        assert bool(torch.isfinite(dX).all()) and bool(torch.isfinite(dW).all())
        for name, got, want in (("dX", dX, dx), ("dW", dW, dw), ("db", db, dbias)):
            ref.check(name, got, want)


def test_large_tiles_and_splits(pg):
    """The scales in every kind of product: whole and split tiles of all sizes, few rows, two steps of rows."""
    for M, N, K in ((2050, 4098, 520), (600, 1030, 2062), (8250, 1004, 24), (20, 3001, 1100)):
        say("sizes", (M, N, K))
        gen = torch.Generator(device="cuda").manual_seed(M)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        rows = 2.0 ** (torch.arange(M, device="cuda") % 23 - 13).float()
        dH, U, G = (rows[:, None] * rnd(M, N)).to(F16), (30 * rnd(M, N)).to(F16), rnd(M, N).to(F16)
        X = rnd(M, K).to(F16)
        Wg, Wu = ((rnd(N, K) * 2.0 ** -8).to(F16).t() for _ in range(2))
        old, ref.WHERE = ref.WHERE, "cuda"
        try:
            for order in ("kn", "nk"):
                check_gated(pg, dH, X, Wg, Wu, G, U, "gelu_tanh", torch.float32, order)
        finally:
            ref.WHERE = old


def test_each_gradient_alone_equals_all_of_them(pg):
    M, N, K = 130, 200, 72
    say("alone")
    gen = torch.Generator().manual_seed(4)
    dH, U, G, X = gpu16(40 * randn(gen, M, N)), gpu16(40 * randn(gen, M, N)), gpu16(randn(gen, M, N)), gpu16(randn(gen, M, K))
    Wg, Wu = (gpu16(randn(gen, K, N) * 2.0 ** -8) for _ in range(2))
    whole = run_gated(pg, dH, X, Wg, Wu, G, U, "silu", torch.float32, "kn")
    for keys in (("dX",), ("dWg", "dWu"), ("dbias_g",), ("dbias_u",), ("dX", "dbias_u")):
        part = {k: torch.empty_like(whole[k]) for k in keys}
        pg.gated_backward(dH, X, Wg, Wu, G, U, act="silu", **part)
        torch.cuda.synchronize()
        for k in keys:
            assert torch.equal(part[k], whole[k]), k


def test_nan_and_infinity_stay_in_their_rows_and_columns(pg):
    """An infinity or NaN among the gradients leaves the other rows of dX and columns of dW as they were."""
    M, N, K = 140, 136, 64
    say("nan")
    gen = torch.Generator().manual_seed(6)
    dH, U, G, X = gpu16(40 * randn(gen, M, N)), gpu16(40 * randn(gen, M, N)), gpu16(randn(gen, M, N)), gpu16(randn(gen, M, K))
    Wg, Wu = (gpu16(randn(gen, K, N) * 2.0 ** -8) for _ in range(2))
    clean = run_gated(pg, dH, X, Wg, Wu, G, U, "silu", torch.float32, "kn")
    for bad in (float("nan"), float("inf"), float("-inf")):
        d = dH.clone()
        d[37, 101] = bad
        got = run_gated(pg, d, X, Wg, Wu, G, U, "silu", torch.float32, "kn")
        assert not bool(torch.isfinite(got["dX"][37]).any())
        keep = torch.arange(M, device="cuda") != 37
        assert torch.equal(got["dX"][keep], clean["dX"][keep])
        keep = torch.arange(N, device="cuda") != 101
        for k in ("dWg", "dWu"):
            assert not bool(torch.isfinite(got[k][:, 101]).any())
            # the clean row 37 of these columns stays: only the entry at 101 changed
            assert torch.equal(got[k][:, keep], clean[k][:, keep])
        for k in ("dbias_g", "dbias_u"):
            assert not bool(torch.isfinite(got[k][101])) and torch.equal(got[k][keep], clean[k][keep])


def test_rows_and_columns_of_zeros(pg):
    M, N, K = 64, 80, 32
    say("zeros")
    gen = torch.Generator().manual_seed(8)
    dH, U, G, X = gpu16(randn(gen, M, N)), gpu16(randn(gen, M, N)), gpu16(randn(gen, M, N)), gpu16(randn(gen, M, K))
    Wg, Wu = (gpu16(randn(gen, K, N)) for _ in range(2))
    dH[5], dH[:, 7] = 0, 0
    got, _ = check_gated(pg, dH, X, Wg, Wu, G, U, "silu", torch.float32, "nk")
    assert bool((got["dX"][5] == 0).all()) and bool((got["dWg"][:, 7] == 0).all()) and bool((got["dWu"][:, 7] == 0).all())
    dH.zero_()
    got = run_gated(pg, dH, X, Wg, Wu, G, U, "silu", F16, "kn")
    assert all(bool((t == 0).all()) for t in got.values())


def test_graph_replays_with_other_ranges(pg):
    """A captured backward pass computes its scales anew from what the inputs hold at each replay."""
    M, N, K = 300, 264, 136
    say("graph")
    gen = torch.Generator().manual_seed(10)
    U, G, X = gpu16(randn(gen, M, N)), gpu16(randn(gen, M, N)), gpu16(randn(gen, M, K))
    Wg, Wu = (gpu16(randn(gen, K, N) * 2.0 ** -6) for _ in range(2))
    base = randn(gen, M, N)
    dH = gpu16(base)
    out = dict(dX=torch.empty(M, K, dtype=F16, device="cuda"), dWg=torch.empty(K, N, device="cuda"),
               dWu=torch.empty(K, N, device="cuda"), dbias_g=torch.empty(N, device="cuda"))
    ws = torch.empty(pg.pgemm_gated_backward_workspace(M, N, K, 1), dtype=torch.uint8, device="cuda")
    pg.gated_backward(dH, X, Wg, Wu, G, U, workspace=ws, **out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pg.gated_backward(dH, X, Wg, Wu, G, U, workspace=ws, **out)
    for rep, scale in enumerate((1.0, 1e4, 1e-6, 1.0, 3e3)):
        dH.copy_(gpu16(base * scale))
        eager = {k: torch.empty_like(v) for k, v in out.items()}
        pg.gated_backward(dH, X, Wg, Wu, G, U, **eager)
        for v in out.values():
            v.fill_(7.0)
        ws.fill_(rep)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], eager[k]), (rep, k)
