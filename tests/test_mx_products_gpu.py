"""Every compiled kernel of the microscaled products on the GPU, and the calls around them: bad scales,
other streams and devices, captured graphs, wide rows, repeats, and the operators as a block uses them."""
import pytest
import torch

import mx_reference as ref
from mx_shapes import EDGES, SHAPES
from software_pipelined_tiled_loop_amd import binding as pg

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def stored(g, rows, K, form, scale=1.0):
    """Random blocks, and their values in 64 bits (of all stored entries) from the operator that is tested elsewhere."""
    mx = pg.mx_quantize(torch.randn(rows, K, generator=g, device="cuda").mul_(scale), pg.mx_empty(rows, K, form, "cuda"))
    return mx, pg.mx_dequantize(mx, torch.empty(rows, ref.filled(K), device="cuda")).double()


def at_once(got, v, e, what):
    d = (got.double() - v).abs()
    bad = ~(d <= e)
    assert not bool(bad.any()), "%s: %d of %d off, the worst by %.3g of its bound at %s" % (
        what, int(bad.sum()), d.numel(), float((d / e.clamp_min(1e-300)).nan_to_num(float("inf")).max()),
        bad.nonzero()[0].tolist())


@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M,N,K", SHAPES + EDGES)
def test_every_kernel(M, N, K, form):
    g = gen(M * 31 + N * 7 + K)
    X, x = stored(g, M, K, form)
    Wg, wg = stored(g, N, K, "mx4", K ** -0.5)
    Wu, wu = stored(g, N, K, "mx4", K ** -0.5)
    for t in TYPES.values():
        zg, eg = ref.product(x, wg, form, t)
        zu, eu = ref.product(x, wu, form, t)
        Y = pg.mx_linear(X, Wg, torch.full((M, N + 1), 9.0, dtype=t, device="cuda")[:, :N])
        at_once(Y, *ref.round_out(zg, eg, t), "linear %s" % t)
        b, R = torch.randn(N, generator=g, device="cuda").to(t), torch.randn(M, N, generator=g, device="cuda").to(t)
        Y = pg.mx_linear(X, Wg, torch.empty(M, N, dtype=t, device="cuda"), bias=b, residual=R, act="gelu_tanh")
        z = zg + b.double()
        v, ev = ref.act_bound(z, eg + 2 * ref.S * (z.abs() + b.double().abs()), "gelu_tanh")
        v = v + R.double()
        at_once(Y, *ref.round_out(v, ev + ref.S * (v.abs() + ev), t), "linear with all %s" % t)
        H = pg.mx_gated(X, Wg, Wu, torch.full((M, N + 8), 9.0, dtype=t, device="cuda")[:, :N])
        v, ev = ref.act_bound(zg, eg, "silu")
        h = v * zu
        at_once(H, *ref.round_out(h, ev * zu.abs() + v.abs() * eu + ev * eu + ref.S * h.abs(), t), "gated %s" % t)
        assert bool((H.as_strided((M, 8), (N + 8, 1), N)[:-1] == 9).all())


# one row of few, a few-rows kernel of several tiles, 128- and 256-row tiles, and (fp32, MX8) the values' way
PLACES = [(1, 64, 512), (40, 200, 1300), (300, 700, 900), (2304, 2297, 1100)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M,N,K", PLACES)
def test_bad_scales_and_entries_stay_in_their_rows(M, N, K, form, dtype):
    """A NaN scale or entry makes its row of the output NaN, a weight's its column; no other value changes."""
    t, g = TYPES[dtype], gen(5)
    X, _ = stored(g, M, K, form)
    W, _ = stored(g, N, K, "mx4")
    clean = pg.mx_linear(X, W, torch.empty(M, N, dtype=t, device="cuda"))
    m, n = M // 2, N - 3
    X[1][m, (K // 2) // 32] = 255
    if form == "mx8" and M > 1:
        X[0][M - 1, K - 1] = 127
    W[1][n, 0] = 255
    Y = pg.mx_linear(X, W, torch.empty(M, N, dtype=t, device="cuda"))
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[m] = True
    bad[:, n] = True
    if form == "mx8" and M > 1:
        bad[M - 1] = True
    assert torch.equal(Y.isnan(), bad)
    assert torch.equal(Y[~bad], clean[~bad])


@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M,N,K", PLACES)
def test_scales_over_their_range(M, N, K, form):
    """Blocks of very different sizes, the smallest scales among them."""
    g = gen(6)
    size = torch.ldexp(torch.ones((), device="cuda"), torch.randint(-60, 30, (M, K // 20 + 1), generator=g, device="cuda"))
    X = pg.mx_quantize(torch.randn(M, K, generator=g, device="cuda") * size.repeat_interleave(20, 1)[:, :K],
                       pg.mx_empty(M, K, form, "cuda"))
    W, w = stored(g, N, K, "mx4", 2.0 ** -20)
    x = pg.mx_dequantize(X, torch.empty(M, ref.filled(K), device="cuda")).double()
    for t in (torch.float32, torch.bfloat16):
        z, e = ref.product(x, w, form, t)
        at_once(pg.mx_linear(X, W, torch.empty(M, N, dtype=t, device="cuda")), *ref.round_out(z, e, t), str(t))


@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M", [5, 300, 2304])
def test_the_smallest_entries(M, form):
    """Entries below 2^-126, down to 2^-133, with weights that bring the products back: nothing is taken for zero."""
    g, N, K = gen(12), 2297 if M > 300 else 70, 512
    X, W = pg.mx_empty(M, K, form, "cuda"), pg.mx_empty(N, K, "mx4", "cuda")
    codes = torch.randint(0, 256, X[0].shape, generator=g, device="cuda")
    X[0].copy_(torch.where(codes % 128 == 127, torch.zeros_like(codes), codes) if form == "mx8" else codes)  # no NaN
    X[1].copy_(torch.randint(3, 9, X[1].shape, generator=g, device="cuda"))
    W[0].copy_(torch.randint(0, 256, W[0].shape, generator=g, device="cuda"))
    W[1].copy_(torch.randint(220, 224, W[1].shape, generator=g, device="cuda"))
    x, w = ref.values(*X, form).cuda(), ref.values(*W, "mx4").cuda()
    for t in (torch.float32, torch.bfloat16):
        z, e = ref.product(x, w, form, t)
        at_once(pg.mx_linear(X, W, torch.empty(M, N, dtype=t, device="cuda")), *ref.round_out(z, e, t), str(t))
    back = pg.mx_dequantize(X, torch.empty(M, K, device="cuda"))
    assert torch.equal(back.double(), x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", PLACES)
def test_streams_graphs_and_repeats(M, N, K, dtype):
    """The same call again, on another stream, and two graphs of it replayed in turn among other work: the same results."""
    t, g = TYPES[dtype], gen(7)
    K = 8200 if M < 100 else K  # contractions that are split
    X, _ = stored(g, M, K, "mx8")
    Wg, _ = stored(g, N, K, "mx4", K ** -0.5)
    Wu, _ = stored(g, N, K, "mx4", K ** -0.5)
    weight = torch.randn(N, generator=g, device="cuda").to(t)

    def run(out):
        H, Y, y = out
        pg.mx_gated(X, Wg, Wu, H)
        pg.mx_linear(X, Wg, Y, residual=H, act="silu")
        pg.rms_norm(Y, weight, y, residual=H)

    fresh = lambda: [torch.zeros(M, N, dtype=t, device="cuda") for _ in range(3)]  # noqa: E731
    want, got = fresh(), fresh()
    run(want)
    run(got)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    other, got = torch.cuda.Stream(), fresh()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        run(got)
    torch.cuda.current_stream().wait_stream(other)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    sets, graphs = [fresh(), fresh()], [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for out, graph in zip(sets, graphs):
        with torch.cuda.graph(graph):
            run(out)
    for turn in range(4):
        for out in sets:
            for o in out:
                o.zero_()
        graphs[turn % 2].replay()
        got = fresh()
        run(got)  # eager work between the replays
        graphs[1 - turn % 2].replay()
        torch.cuda.synchronize()
        for out in sets + [got]:
            assert all(torch.equal(a, b) for a, b in zip(want, out)), turn
    # other contents behind the same addresses: nothing is kept from the capture
    X[0].copy_(X[0].roll(1, 0) ^ 128)
    run(want)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for out in sets:
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_offsets_beyond_32_bits():
    """Rows so far apart that the last ones lie beyond 2^31 and 2^32 bytes, in each operand in turn."""
    K, N, far, big = 512, 96, 1 << 20, 5000
    g = gen(8)
    W, _ = stored(g, N, K, "mx4")
    space = torch.zeros(5001 * far, dtype=torch.uint8, device="cuda")

    def apart(rows, width, by, dtype=torch.uint8):
        return space.view(dtype).as_strided((rows, width), (by // torch.empty((), dtype=dtype).element_size(), 1))

    Xb, _ = stored(g, big, K, "mx8")
    q = apart(big, 512, far)
    q.copy_(Xb[0])
    full = pg.mx_linear(Xb, W, torch.empty(big, N, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(pg.mx_linear((q, Xb[1]), W, torch.empty(big, N, dtype=torch.bfloat16, device="cuda")), full)
    Y = apart(big, N, far, torch.bfloat16)
    assert torch.equal(pg.mx_linear(Xb, W, Y), full)
    x = apart(big, K, far, torch.bfloat16)
    x.copy_(torch.randn(big, K, generator=g, device="cuda"))
    w = torch.randn(K, generator=g, device="cuda").bfloat16()
    assert torch.equal(pg.rms_norm(x, w, torch.empty(big, K, dtype=torch.bfloat16, device="cuda")),
                       pg.rms_norm(x.contiguous(), w, torch.empty(big, K, dtype=torch.bfloat16, device="cuda")))
    a, b = pg.mx_quantize(x, pg.mx_empty(big, K, "mx4", "cuda")), pg.mx_quantize(x.contiguous(), pg.mx_empty(big, K, "mx4", "cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = x.t().contiguous().t()  # columns
    b = pg.mx_quantize(c, pg.mx_empty(big, K, "mx4", "cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dense = pg.mx_dequantize(a, torch.empty(big, K, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(pg.mx_dequantize(a, x), dense)
    dy = torch.randn(big, K, generator=g, device="cuda").bfloat16()
    outs = []
    for place in (apart(big, K, far, torch.bfloat16), torch.empty(big, K, dtype=torch.bfloat16, device="cuda")):
        dw = torch.empty(K, dtype=torch.bfloat16, device="cuda")
        pg.rms_norm_backward(dy, dense, w, dX=place, dweight=dw)
        outs.append((place, dw))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M,N", [(2, 7), (300, 130), (2304, 2297)])
def test_no_entries(M, N, form, dtype):
    """K = 0 on every way: bias, activation and residual alone."""
    t, g = TYPES[dtype], gen(M)
    X, W = pg.mx_empty(M, 0, form, "cuda"), pg.mx_empty(N, 0, "mx4", "cuda")
    b, u = (torch.randn(N, generator=g, device="cuda").to(t) for _ in range(2))
    R = torch.randn(M, N, generator=g, device="cuda").to(t)
    assert torch.equal(pg.mx_linear(X, W, torch.full_like(R, 9)), torch.zeros_like(R))
    assert torch.equal(pg.mx_linear(X, W, torch.full_like(R, 9), bias=b, residual=R, act="relu"),
                       (b.float().clamp_min(0) + R.float()).to(t))
    assert torch.equal(pg.mx_gated(X, W, W, torch.full_like(R, 9), bias_g=b, bias_u=u, act="relu"),
                       (b.float().clamp_min(0) * u.float()).to(t).expand(M, N))


def test_far_rows_of_large_tiles():
    """The large tiles' own epilogue, output and residual beyond 2^32 bytes, at the output's odd edges."""
    M, N, K, far = 4600, 3507, 300, 1 << 20
    g = gen(9)
    X, _ = stored(g, M, K, "mx4")
    W, _ = stored(g, N, K, "mx4", K ** -0.5)
    near = torch.randn(M, N, generator=g, device="cuda").bfloat16()
    space = torch.full((M * far // 2,), 9.0, dtype=torch.bfloat16, device="cuda")
    R, Y = (space.as_strided((M, N), (far // 2, 1), at) for at in (5, 8200))
    R.copy_(near)
    want = pg.mx_linear(X, W, torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), residual=near, act="silu")
    assert torch.equal(pg.mx_linear(X, W, Y, residual=R, act="silu"), want)
    assert torch.equal(R, near)
    assert bool((space.as_strided((M, 8200 - 5 - N), (far // 2, 1), 5 + N) == 9).all())
    assert bool((space.as_strided((M, far // 2 - 8200 - N), (far // 2, 1), 8200 + N) == 9).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N", [(5, 700), (3, 5000), (2, 20001)])
def test_norms_in_place(M, N, dtype):
    """h over x or over the residual, dx over dh: the same results."""
    t, g = TYPES[dtype], gen(N)
    x, r, dy, dh = (torch.randn(M, N, generator=g, device="cuda").to(t) for _ in range(4))
    w = torch.randn(N, generator=g, device="cuda").to(t)
    h, y = torch.empty_like(x), torch.empty_like(x)
    pg.rms_norm(x, w, y, residual=r, H=h)
    for k in range(2):
        a = [x.clone(), r.clone()]
        again = torch.empty_like(y)
        pg.rms_norm(a[0], w, again, residual=a[1], H=a[k])
        assert torch.equal(again, y) and torch.equal(a[k], h)
    dx, dw = pg.rms_norm_backward(dy, h, w, dH=dh, dX=torch.empty_like(x), dweight=torch.empty_like(w))
    over = dh.clone()
    dw2 = torch.empty_like(w)
    pg.rms_norm_backward(dy, h, w, dH=over, dX=over, dweight=dw2)
    assert torch.equal(over, dx) and torch.equal(dw2, dw)


def test_norm_gradient_against_differences():
    """The backward pass against central differences of the forward pass: they differ by what the 64-bit forms say (the
    differences' own cubic term) and by the roundings of both passes, as bounded there."""
    g = gen(11)
    M, N, step, t = 4, 65, 2.0 ** -6, torch.float32
    h, dy, w = (torch.randn(*s, generator=g, device="cuda") for s in ((M, N), (M, N), (N,)))
    dx, dw = pg.rms_norm_backward(dy, h, w, dX=torch.empty_like(h), dweight=torch.empty_like(w))
    (wx, ex), (ww, ew) = ref.norm_backward(dy, h, w, None, 1e-6)
    (wx, ex), (ww, ew) = ref.round_out(wx, ex, t), ref.round_out(ww, ew, t)
    d64 = dy.double().cpu()

    def loss(h_, w_):
        """(of the operator, of the 64-bit form, how far apart they may be)"""
        y = pg.rms_norm(h_, w_, torch.empty_like(h_)).double().cpu()
        v, e = ref.round_out(*ref.norm(h_, None, w_, 1e-6)[1], t)
        return (y * d64).sum(), (v * d64).sum(), (e * d64.abs()).sum()
    for _ in range(12):
        vh, vw = torch.randn(M, N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
        for up, down, v, got, want, e in ((loss(h + step * vh, w), loss(h - step * vh, w), vh, dx, wx, ex),
                                          (loss(h, w + step * vw), loss(h, w - step * vw), vw, dw, ww, ew)):
            v = v.double().cpu()
            difference, plain = (up[0] - down[0]) / (2 * step), (up[1] - down[1]) / (2 * step)
            cubic = plain - (want * v).sum()
            bound = (up[2] + down[2]) / (2 * step) + (e * v.abs()).sum()
            # (h +- step v is rounded, the same way in both forms: half the difference's slope errs by 2^-24 of |h| or |w|)
            rounding = 2.0 ** -24 * (want.abs() * ((h if v.dim() == 2 else w).double().cpu().abs() + step * v.abs())).sum() / step
            assert abs(difference - cubic - (got.double().cpu() * v).sum()) <= bound + 4 * rounding
            assert abs(cubic) < 0.1 * (want.abs() * v.abs()).sum()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M", [1, 33, 300])
def test_a_block_as_it_is_used(M, form, dtype):
    """norm -> blocks -> gated -> blocks -> linear with the residual -> norm, each step against its plain form."""
    t, g = TYPES[dtype], gen(M)
    N, D, eps = 264, 700, 1e-5
    x, r = (torch.randn(M, N, generator=g, device="cuda").to(t) for _ in range(2))
    w1, w2 = (torch.randn(N, generator=g, device="cuda").to(t) for _ in range(2))
    Wg, Wu = stored(g, D, N, "mx4", N ** -0.5)[0], stored(g, D, N, "mx4", N ** -0.5)[0]
    Wd = stored(g, N, D, "mx4", D ** -0.5)[0]
    h, X = torch.empty(M, N, dtype=t, device="cuda"), pg.mx_empty(M, N, form, "cuda")
    pg.rms_norm(x, w1, residual=r, H=h, mx=X, eps=eps)
    (wh, eh), (wy, ey) = ref.norm(x, r, w1, eps)
    ref.close(h, ref.round_out(wh, eh, t), "residual stream")
    ref.check_blocks(X, wy, ey, "blocks of the norm")
    a = pg.mx_gated(X, Wg, Wu, torch.empty(M, D, dtype=t, device="cuda"))
    ref.close(a, ref.gated(X, Wg, Wu, None, None, "silu", t), "gated")
    A = pg.mx_quantize(a, pg.mx_empty(M, D, form, "cuda"))
    want = ref.quantize(a, form)
    assert torch.equal(A[0].cpu(), want[0]) and torch.equal(A[1].cpu(), want[1])
    old = h.clone()
    pg.mx_linear(A, Wd, h, residual=h)
    ref.close(h, ref.linear(A, Wd, None, old, "none", t), "linear onto the residual stream")
    y = pg.rms_norm(h, w2, torch.empty_like(h), eps=eps)
    ref.close(y, ref.round_out(*ref.norm(h, None, w2, eps)[1], t), "last norm")
    # and back through the norm
    dy, dx, dw = torch.randn(M, N, generator=g, device="cuda").to(t), torch.empty_like(h), torch.empty_like(w2)
    pg.rms_norm_backward(dy, h, w2, dX=dx, dweight=dw, eps=eps)
    (wx, ex), (ww, ew) = ref.norm_backward(dy, h, w2, None, eps)
    ref.close(dx, ref.round_out(wx, ex, t), "dx")
    ref.close(dw, ref.round_out(ww, ew, t), "dw")
