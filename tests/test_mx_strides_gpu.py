"""The microscaled operators on blocks whose rows lie apart, at the least alignment that the entries take, and in 4 bits
again and again, on another stream and in graphs; the residual in place on every kind of tile."""
import pytest
import torch

import mx_reference as ref
from mx_cut_shapes import PLACES
from software_pipelined_tiled_loop_amd import binding as pg

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def blocks(g, rows, K, form, scale=1.0):
    return pg.mx_quantize(torch.randn(rows, K, generator=g, device="cuda").mul_(scale), pg.mx_empty(rows, K, form, "cuda"))


def apart(t, gap, first, fill):
    """A matrix of bytes as rows `gap` bytes apart, from byte `first` of its memory on; `fill` everywhere else."""
    rows, width = t.shape
    space = torch.full((first + rows * (width + gap),), fill, dtype=torch.uint8, device="cuda")
    return space, space.as_strided((rows, width), (width + gap, 1), first)


def spread(mx, gaps=(16, 4)):
    """The same blocks with rows apart; what lies between them are NaN scales and entries."""
    out = []
    for t, gap in zip(mx, gaps):
        _, s = apart(t, gap, gap, 255)
        out.append(s.copy_(t))
    return tuple(out)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M,N,K", [(1, 64, 8200)] + PLACES)
def test_rows_of_blocks_apart(M, N, K, form, dtype):
    """Codes 16 bytes and scales 4 bytes further apart than they are long: the dense calls' bits."""
    t, g = TYPES[dtype], gen(M + N)
    X, Wg, Wu = blocks(g, M, K, form), blocks(g, N, K, "mx4", K ** -0.5), blocks(g, N, K, "mx4", K ** -0.5)
    b, R = torch.randn(N, generator=g, device="cuda").to(t), torch.randn(M, N, generator=g, device="cuda").to(t)
    fresh = lambda: torch.full((M, N), 9.0, dtype=t, device="cuda")  # noqa: E731
    y = pg.mx_linear(X, Wg, fresh(), bias=b, residual=R, act="silu")
    h = pg.mx_gated(X, Wg, Wu, fresh())
    assert bool(y.isfinite().all()) and bool(h.isfinite().all())
    for gaps in ((16, 4), (48, 12), (0, 4)):
        x, wg, wu = spread(X, gaps), spread(Wg, gaps), spread(Wu, gaps)
        assert torch.equal(pg.mx_linear(x, wg, fresh(), bias=b, residual=R, act="silu"), y), gaps
        assert torch.equal(pg.mx_linear(X, wg, fresh(), bias=b, residual=R, act="silu"), y), gaps
        assert torch.equal(pg.mx_gated(x, wg, wu, fresh()), h), gaps
        assert torch.equal(pg.mx_gated(x, Wg, Wu, fresh()), h), gaps


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("R,K", [(1, 300), (70, 257), (129, 4001), (3, 16500)])
def test_blocks_are_written_apart(R, K, form, dtype):
    """Rows and columns quantised, and the norm's blocks, into rows apart: the dense blocks, nothing between them."""
    t, g = TYPES[dtype], gen(R + K)
    x, w = torch.randn(R, K, generator=g, device="cuda").to(t), torch.randn(K, generator=g, device="cuda").to(t)
    turned = x.t().contiguous().t()
    for write in (lambda m: pg.mx_quantize(x, m), lambda m: pg.mx_quantize(turned, m), lambda m: pg.rms_norm(x, w, mx=m)):
        want = write(pg.mx_empty(R, K, form, "cuda"))
        spaces, got = zip(*(apart(m, gap, gap, 7) for m, gap in zip(want, (16, 4))))
        write(got)
        for space, a, b, gap in zip(spaces, got, want, (16, 4)):
            assert torch.equal(a, b)
            between = space.as_strided((R + 1, gap), (a.shape[1] + gap, 1), 0)  # (before each row, and behind the last)
            assert bool((between == 7).all())
        back = [pg.mx_dequantize(m, torch.empty(R, K, device="cuda")) for m in (got, want)]
        assert torch.equal(*back)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M,N,K", [(1, 64, 8200)] + PLACES)
def test_residual_in_place(M, N, K, form, dtype):
    t, g = TYPES[dtype], gen(M + K)
    X, W = blocks(g, M, K, form), blocks(g, N, K, "mx4", K ** -0.5)
    wide = torch.randn(M, N + 3, generator=g, device="cuda").to(t)
    R = wide[:, :N]
    for act in ("none", "gelu"):
        want = pg.mx_linear(X, W, torch.empty(M, N, dtype=t, device="cuda"), residual=R, act=act)
        again = wide.clone()
        pg.mx_linear(X, W, again[:, :N], residual=again[:, :N], act=act)
        assert torch.equal(again[:, :N], want) and torch.equal(again[:, N:], wide[:, N:])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N,K", [(1, 64, 8200)] + PLACES)
def test_streams_graphs_and_repeats_in_4_bits(M, N, K, dtype):
    """The same calls again, on another stream, and two graphs of them replayed in turn among other work: the same bits."""
    t, g = TYPES[dtype], gen(7)
    X = blocks(g, M, K, "mx4")
    Wg, Wu = blocks(g, N, K, "mx4", K ** -0.5), blocks(g, N, K, "mx4", K ** -0.5)
    weight = torch.randn(N, generator=g, device="cuda").to(t)

    def run(out):
        H, Y, y, codes, scales = out
        pg.mx_gated(X, Wg, Wu, H)
        pg.mx_linear(X, Wg, Y, residual=H, act="silu")
        pg.rms_norm(Y, weight, y, residual=H, mx=(codes, scales))

    fresh = lambda: [torch.zeros(M, N, dtype=t, device="cuda") for _ in range(3)] + [  # noqa: E731
        m.zero_() for m in pg.mx_empty(M, N, "mx4", "cuda")]
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    want = fresh()
    run(want)
    for _ in range(4):
        got = fresh()
        run(got)
        assert same(want, got)
    other, got = torch.cuda.Stream(), fresh()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        run(got)
    torch.cuda.current_stream().wait_stream(other)
    assert same(want, got)
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
            assert same(want, out), turn
    # other contents behind the same addresses: nothing is kept from the capture
    X[0].copy_(X[0].roll(1, 1) ^ 8)
    run(want)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for out in sets:
        assert same(want, out)


@pytest.mark.parametrize("form", ["mx8", "mx4"])
def test_a_product_against_its_form_on_rows_apart(form):
    """(the dense calls are checked elsewhere; here one of each tile straight against 64 bits)"""
    for M, N, K in PLACES:
        g = gen(M * 3 + N)
        X, W = blocks(g, M, K, form), blocks(g, N, K, "mx4", K ** -0.5)
        v = [pg.mx_dequantize(m, torch.empty(m[0].shape[0], ref.filled(K), device="cuda")).double() for m in (X, W)]
        for t in TYPES.values():
            z, e = ref.round_out(*ref.product(*v, form, t), t)
            got = pg.mx_linear(spread(X), spread(W), torch.empty(M, N, dtype=t, device="cuda"))
            assert bool(((got.double() - z).abs() <= e).all()), (M, N, K, t)
