"""The feed-forward operators on the GPU against their 64-bit forms.

Sizes run over one token, odd and ragged extents, contractions shorter and
longer than a K tile, split sums and empty sizes; operands over types, storage
orders, padded rows and misaligned bases.  Padding holds NaN and outputs start
as a sentinel, so a read or write out of place shows.  The bounds are derived
in linear_reference.py.  Every case prints itself before it runs.
"""
import itertools

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SENTINEL = 77.0


@pytest.fixture(scope="module")
def pg():
    from software_pipelined_tiled_loop_amd import binding
    return binding


class Maker:
    """Seeded operands inside larger buffers: NaN around inputs, a sentinel around outputs."""

    def __init__(self, seed, dtype, pad=0, shift=0, device="cuda"):
        self.gen = torch.Generator()
        self.gen.manual_seed(seed)
        self.dtype, self.pad, self.shift, self.device = dtype, pad, shift, device
        self.outs = []

    def _frame(self, r, c, dtype, fill):
        ld = c + self.pad
        whole = torch.full((self.shift + r * ld + 16,), fill, dtype=dtype, device=self.device)
        return whole, whole[self.shift:self.shift + r * ld].view(r, ld)[:, :c]

    def rows(self, r, c, scale=1.0, dtype=None):
        _, v = self._frame(r, c, dtype or self.dtype, float("nan"))
        v.copy_((torch.randn(r, c, generator=self.gen) * scale).to(dtype or self.dtype))
        return v

    def weight(self, k, n, order, dtype=None):
        s = max(k, 1) ** -0.5
        return self.rows(k, n, s, dtype) if order == "kn" else self.rows(n, k, s, dtype).t()

    def vector(self, n):
        return self.rows(1, n, 0.5)[0]

    def out(self, r, c, dtype=None):
        whole, v = self._frame(r, c, dtype or self.dtype, SENTINEL)
        self.outs.append((whole, v))
        return v

    def weight_out(self, k, n, order, dtype=None):
        return self.out(k, n, dtype) if order == "kn" else self.out(n, k, dtype).t()

    def vector_out(self, n, dtype=None):
        return self.out(1, n, dtype)[0]

    def check_frames(self):
        """Nothing outside an output was written (call after reading the outputs)."""
        for whole, v in self.outs:
            v.fill_(SENTINEL)
            assert bool((whole == SENTINEL).all()), "written outside the output"


def say(*a):
    print("[case]", *a, flush=True)


#            M     N     K
FORWARD = [(1, 1, 1), (1, 64, 64), (1, 4100, 136), (2, 9, 7), (3, 7, 130), (16, 128, 256), (17, 33, 65), (32, 96, 1000),
           (48, 250, 2049), (64, 8, 512), (65, 40, 96), (128, 128, 64), (129, 257, 100), (257, 511, 200), (300, 64, 1032),
           (1, 5, 3000), (5, 1, 4096)]


def options(i):
    """Acts, flags and layouts walk through their combinations with the case's number."""
    return dict(act=ref.ACTS[i % 5], bias=i % 2 == 0, residual=i % 3 != 1, keep=i % 4 < 2, pad=(0, 1, 8)[i % 3],
                shift=(0, 1, 3)[(i // 2) % 3], f32_out=i % 5 == 3)


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("i", range(len(FORWARD)))
def test_linear(pg, dtype, order, i):
    M, N, K = FORWARD[i]
    o = options(i + (order == "nk") * 2 + len(dtype))
    say("linear", dtype, order, (M, N, K), o)
    t = TYPES[dtype]
    yt = torch.float32 if o["f32_out"] else t
    m = Maker(100 + i, t, o["pad"], o["shift"])
    X, W = m.rows(M, K), m.weight(K, N, order)
    b = m.vector(N) if o["bias"] else None
    R = m.rows(M, N, dtype=yt) if o["residual"] else None
    Y, Z = m.out(M, N, yt), m.out(M, N) if o["keep"] else None
    assert pg.linear(X, W, Y, bias=b, residual=R, act=o["act"], Z=Z) is Y
    torch.cuda.synchronize()
    y, z = ref.linear(X, W, b, R, o["act"], yt)
    ref.check("Y", Y, y)
    if Z is not None:
        ref.check("Z", Z, z)
    m.check_frames()


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("i", range(len(FORWARD)))
def test_gated(pg, dtype, order, i):
    M, N, K = FORWARD[i]
    o = options(i + (order == "nk") * 3 + len(dtype))
    say("gated", dtype, order, (M, N, K), o)
    t = TYPES[dtype]
    ht = torch.float32 if o["f32_out"] else t
    m = Maker(200 + i, t, o["pad"], o["shift"])
    X, Wg, Wu = m.rows(M, K), m.weight(K, N, order), m.weight(K, N, order)
    bg, bu = (m.vector(N) if o["bias"] else None), (m.vector(N) if o["residual"] else None)
    H = m.out(M, N, ht)
    G, U = (m.out(M, N) if o["keep"] else None), (m.out(M, N) if i % 4 != 1 else None)
    assert pg.gated(X, Wg, Wu, H, bias_g=bg, bias_u=bu, act=o["act"], G=G, U=U) is H
    torch.cuda.synchronize()
    h, g, u = ref.gated(X, Wg, Wu, bg, bu, o["act"], ht)
    ref.check("H", H, h)
    for name, got, want in (("G", G, g), ("U", U, u)):
        if got is not None:
            ref.check(name, got, want)
    m.check_frames()


BACKWARD = [(1, 1, 1), (1, 40, 24), (2, 9, 7), (7, 3, 130), (33, 65, 17), (64, 128, 128), (65, 129, 257), (200, 100, 300),
            (520, 36, 50), (1000, 8, 64), (3000, 70, 33), (130, 1040, 16)]


@pytest.mark.parametrize("orders", [("kn", "kn"), ("nk", "nk"), ("kn", "nk")])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("i", range(len(BACKWARD)))
def test_linear_backward(pg, dtype, orders, i):
    M, N, K = BACKWARD[i]
    o = options(i + len(dtype) + (orders[0] != orders[1]))
    say("linear_backward", dtype, orders, (M, N, K), o)
    t = TYPES[dtype]
    gt = torch.float32 if o["f32_out"] else t
    m = Maker(300 + i, t, o["pad"], o["shift"])
    dY, X, W, Z = m.rows(M, N), m.rows(M, K), m.weight(K, N, orders[0]), m.rows(M, N)
    dX, dW = m.out(M, K), m.weight_out(K, N, orders[1], gt)
    db = m.vector_out(N, gt) if o["bias"] else None
    pg.linear_backward(dY, X, W, Z=Z if o["act"] != "none" else None, act=o["act"], dX=dX, dW=dW, dbias=db)
    torch.cuda.synchronize()
    dx, dw, dbias = ref.linear_backward(dY, X, W, Z, o["act"], gt)
    ref.check("dX", dX, dx)
    ref.check("dW", dW, dw)
    if db is not None:
        ref.check("dbias", db, dbias)
    m.check_frames()


@pytest.mark.parametrize("orders", [("kn", "kn"), ("nk", "nk"), ("nk", "kn")])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("i", range(len(BACKWARD)))
def test_gated_backward(pg, dtype, orders, i):
    M, N, K = BACKWARD[i]
    o = options(i + len(dtype) + 2 * (orders[0] != orders[1]))
    say("gated_backward", dtype, orders, (M, N, K), o)
    t = TYPES[dtype]
    gt = torch.float32 if o["f32_out"] else t
    m = Maker(400 + i, t, o["pad"], o["shift"])
    dH, X, G, U = m.rows(M, N), m.rows(M, K), m.rows(M, N), m.rows(M, N)
    Wg, Wu = m.weight(K, N, orders[0]), m.weight(K, N, orders[0])
    dX, dWg, dWu = m.out(M, K), m.weight_out(K, N, orders[1], gt), m.weight_out(K, N, orders[1], gt)
    dbg, dbu = (m.vector_out(N, gt) if o["bias"] else None), (m.vector_out(N, gt) if o["keep"] else None)
    pg.gated_backward(dH, X, Wg, Wu, G, U, act=o["act"], dX=dX, dWg=dWg, dWu=dWu, dbias_g=dbg, dbias_u=dbu)
    torch.cuda.synchronize()
    want = ref.gated_backward(dH, X, Wg, Wu, G, U, o["act"], gt)
    for name, got, w in zip(("dX", "dWg", "dWu", "dbg", "dbu"), (dX, dWg, dWu, dbg, dbu), want):
        if got is not None:
            ref.check(name, got, w)
    m.check_frames()


@pytest.mark.parametrize("act", ref.ACTS)
@pytest.mark.parametrize("dtype", list(TYPES))
def test_activations_over_their_range(pg, dtype, act):
    """act and act' from the far negative to the far positive, through a product with the identity."""
    say("range", dtype, act)
    t = TYPES[dtype]
    n = 64
    x = torch.cat([torch.linspace(-12, 12, 64 * 60), torch.tensor([0.0, -0.0, 1e-3, -1e-3, 30, -30, 200, -200, 3e4, -3e4]),
                   torch.zeros(54)])
    Z = x.view(-1, n).to(t).cuda()
    M = Z.shape[0]
    eye = torch.eye(n, dtype=t, device="cuda")
    Y = torch.empty(M, n, dtype=torch.float32, device="cuda")
    pg.linear(Z, eye, Y, act=act)
    ref.check("act", Y, ref.linear(Z, eye, None, None, act, torch.float32)[0])
    one = torch.ones(M, n, dtype=t, device="cuda")
    dX = torch.empty(M, n, dtype=t, device="cuda")
    pg.linear_backward(one, Z, eye, Z=Z, act=act, dX=dX)
    ref.check("slope", dX, ref.linear_backward(one, Z, eye, Z, act, t)[0])


@pytest.mark.parametrize("dtype", list(TYPES))
def test_nan_and_infinity_stay_in_their_rows_and_columns(pg, dtype):
    t = TYPES[dtype]
    say("nan", dtype)
    m = Maker(7, t)
    X, W, R = m.rows(130, 200), m.weight(200, 140, "kn"), m.rows(130, 140)
    X[3, 5] = float("nan")
    X[129, 199] = float("inf")
    W[:, 139] = float("inf")
    for act in ref.ACTS:
        Y = m.out(130, 140)
        pg.linear(X, W, Y, residual=R, act=act)
        y = Y.double().cpu()
        want = ref.act64(d64(X) @ d64(W), act) + d64(R)
        if act in ("gelu", "silu", "gelu_tanh"):
            # act(-inf) is 0 as a limit and NaN as written: either is allowed
            z = d64(X) @ d64(W)
            skip = z == float("-inf")
        else:
            skip = torch.zeros_like(want, dtype=torch.bool)
        assert torch.equal(torch.isfinite(y)[~skip], torch.isfinite(want)[~skip]), act
        assert torch.equal(torch.isnan(y)[~skip], torch.isnan(want)[~skip]), act


@pytest.fixture
def on_gpu(monkeypatch):
    """The 64-bit form evaluated on the GPU (float64 products), for the large sizes."""
    monkeypatch.setattr(ref, "WHERE", "cuda")


#        M     N     K
LARGE = [(2500, 2310, 200), (4096, 2048, 96), (3001, 2999, 65), (1100, 8200, 130), (2304, 2304, 1110)]


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("i", range(len(LARGE)))
def test_large_tiles(pg, on_gpu, dtype, order, i):
    """Sizes that fill the GPU, where the planner takes the large tile, in every layout."""
    M, N, K = LARGE[i]
    say("large", dtype, order, (M, N, K))
    t, act = TYPES[dtype], ref.ACTS[1 + i % 4]
    m = Maker(500 + i, t, (0, 1, 8, 0, 2)[i], (0, 1, 0, 3, 0)[i])
    X, W, Wu = m.rows(M, K), m.weight(K, N, order), m.weight(K, N, order)
    b, R = m.vector(N), m.rows(M, N)
    Y, Z = m.out(M, N), m.out(M, N)
    pg.linear(X, W, Y, bias=b, residual=R, act=act, Z=Z)
    y, z = ref.linear(X, W, b, R, act, t)
    ref.check("Y", Y, y)
    ref.check("Z", Z, z)
    H, G, U = m.out(M, N), m.out(M, N), m.out(M, N)
    pg.gated(X, W, Wu, H, act=act, G=G, U=U)
    for name, got, want in zip("HGU", (H, G, U), ref.gated(X, W, Wu, None, None, act, t)):
        ref.check(name, got, want)
    # the gradients contract over N and over M; dW is K x N
    dX, dW, dWu = m.out(M, K), m.weight_out(K, N, order), m.weight_out(K, N, order)
    pg.gated_backward(R, X, W, Wu, G, U, act=act, dX=dX, dWg=dW, dWu=dWu)
    for name, got, want in zip(("dX", "dWg", "dWu"), (dX, dW, dWu), ref.gated_backward(R, X, W, Wu, G, U, act, t)):
        ref.check(name, got, want)
    # dX of many columns and dW of many rows: the other roles of the large tile
    X2, W2, dY = m.rows(K, N), m.weight(N, M, order), m.rows(K, M)
    dX2, dW2, db = m.out(K, N), m.weight_out(N, M, order), m.vector_out(M)
    pg.linear_backward(dY, X2, W2, dX=dX2, dW=dW2, dbias=db)
    for name, got, want in zip(("dX", "dW", "db"), (dX2, dW2, db), ref.linear_backward(dY, X2, W2, None, "none", t)):
        ref.check(name, got, want)
    m.check_frames()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M", [8200, 8250])
def test_gradients_of_many_rows(pg, on_gpu, dtype, M):
    """Sizes where a workgroup of the slope kernel takes two steps of rows, the last one or both cut."""
    N, K, t = 1004, 24, TYPES[dtype]
    for act in ref.ACTS:
        say("many rows", dtype, M, act)
        m = Maker(700, t, 1, 1)
        dY, X, G, U = m.rows(M, N), m.rows(M, K), m.rows(M, N), m.rows(M, N)
        Wg, Wu = m.weight(K, N, "kn"), m.weight(K, N, "kn")
        dX, dW, db = m.out(M, K), m.weight_out(K, N, "kn"), m.vector_out(N)
        pg.linear_backward(dY, X, Wg, Z=G, act=act, dX=dX, dW=dW, dbias=db)
        for name, got, want in zip(("dX", "dW", "db"), (dX, dW, db), ref.linear_backward(dY, X, Wg, G, act, t)):
            ref.check(name, got, want)
        dWu, dbu = m.weight_out(K, N, "kn"), m.vector_out(N)
        pg.gated_backward(dY, X, Wg, Wu, G, U, act=act, dX=dX, dWg=dW, dWu=dWu, dbias_g=db, dbias_u=dbu)
        for name, got, want in zip(("dX", "dWg", "dWu", "dbg", "dbu"), (dX, dW, dWu, db, dbu),
                                   ref.gated_backward(dY, X, Wg, Wu, G, U, act, t)):
            ref.check(name, got, want)
        m.check_frames()


#       M   N      K     few rows: every width of tile, with and without splits, cut K tiles
FEW = [(1, 4096, 2048), (1, 16384, 520), (3, 33000, 264), (20, 4104, 1000), (40, 4100, 777), (64, 1030, 4001), (17, 300, 9000),
       (33, 8190, 1500)]


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("i", range(len(FEW)))
def test_few_rows(pg, on_gpu, dtype, order, i):
    M, N, K = FEW[i]
    say("few", dtype, order, (M, N, K))
    t, act = TYPES[dtype], ref.ACTS[i % 5]
    m = Maker(600 + i, t, (0, 1, 8)[i % 3], (0, 3, 1)[i % 3])
    X, W, Wu, b, R = m.rows(M, K), m.weight(K, N, order), m.weight(K, N, order), m.vector(N), m.rows(M, N)
    Y, H, U = m.out(M, N), m.out(M, N), m.out(M, N)
    pg.linear(X, W, Y, bias=b, residual=R, act=act)
    ref.check("Y", Y, ref.linear(X, W, b, R, act, t)[0])
    pg.gated(X, W, Wu, H, bias_u=b, act=act, U=U)
    h, _, u = ref.gated(X, W, Wu, None, b, act, t)
    ref.check("H", H, h)
    ref.check("U", U, u)
    dX = m.out(M, K)
    pg.gated_backward(R, X, W, Wu, R, U, act=act, dX=dX)
    ref.check("dX", dX, ref.gated_backward(R, X, W, Wu, R, U, act, t)[0])
    m.check_frames()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ref.ACTS)
def test_activations_at_their_ends(pg, dtype, act):
    """Values whose squares and cubes overflow, infinities and NaN."""
    say("ends", dtype, act)
    t, inf, nan = TYPES[dtype], float("inf"), float("nan")
    x = torch.tensor([3e38, -3e38, 1e20, -1e20, 1e13, -1e13, 1e5, -1e5, 100.0, -100.0, 64.0, -64.0, inf, -inf, nan, 0.0])
    Z = x.view(1, -1).to(t).cuda()
    z = Z.double().cpu()[0]
    eye = torch.eye(16, dtype=t, device="cuda")
    # a product with the identity would turn 0 * inf into NaN: the bias carries the values
    Y, X0 = torch.empty(1, 16, dtype=t, device="cuda"), torch.zeros(1, 16, dtype=t, device="cuda")
    pg.linear(X0, eye, Y, bias=Z[0], act=act)
    y = Y.double().cpu()[0]
    want = torch.where(z > 0, z, torch.zeros_like(z)) if act != "none" else z
    fin = torch.isfinite(z)
    # beyond +-64 act is x or 0; a smooth act of -64 and -100 is below 1e-25
    assert bool(((y - want)[fin].abs() <= ref.half_step(t) * want[fin].abs() + 1e-24).all()), y
    assert y[12] == inf and bool(torch.isnan(y[14]))
    assert y[13] == (-inf if act == "none" else 0.0) or (act in ("silu", "gelu", "gelu_tanh") and bool(torch.isnan(y[13])))
    # slopes: 1 and 0
    one, db = torch.ones(1, 16, dtype=t, device="cuda"), torch.empty(16, dtype=torch.float32, device="cuda")
    pg.linear_backward(one, X0, eye, Z=Z, act=act, dbias=db)
    s = db.double().cpu()
    want = (z > 0).double() if act != "none" else torch.ones(16, dtype=torch.float64)
    want[15] = {"none": 1.0, "relu": 0.0}.get(act, 0.5)
    assert bool(((s - want)[:14].abs() <= 1e-6).all()) and abs(float(s[15] - want[15])) <= 1e-6, s
    if act not in ("none", "relu"):
        assert bool(torch.isnan(s[14]))


def d64(t):
    return t.detach().cpu().double()


@pytest.mark.parametrize("order", ["kn", "nk"])
def test_empty_sizes(pg, order):
    say("empty", order)
    t = torch.bfloat16
    m = Maker(3, t)
    # K = 0: act(bias) + residual
    b, R, Y = m.vector(20), m.rows(5, 20), m.out(5, 20)
    W0 = torch.empty(0, 20, dtype=t, device="cuda") if order == "kn" else torch.empty(20, 0, dtype=t, device="cuda").t()
    X0 = torch.empty(5, 0, dtype=t, device="cuda")
    pg.linear(X0, W0, Y, bias=b, residual=R, act="silu")
    ref.check("Y", Y, ref.linear(X0, W0, b, R, "silu", t)[0])
    # M = 0 or N = 0: nothing forward; zero gradients backward
    X, W = torch.empty(0, 30, dtype=t, device="cuda"), m.weight(30, 20, order)
    pg.linear(X, W, torch.empty(0, 20, dtype=t, device="cuda"))
    dW, db = m.weight_out(30, 20, order), m.vector_out(20)
    e = torch.empty(0, 20, dtype=t, device="cuda")
    pg.linear_backward(e, X, W, Z=e, act="gelu", dX=torch.empty(0, 30, dtype=t, device="cuda"), dW=dW, dbias=db)
    torch.cuda.synchronize()
    assert bool((dW == 0).all()) and bool((db == 0).all())
    Wn = torch.empty(30, 0, dtype=t, device="cuda")
    X5, en, dX = m.rows(5, 30), torch.empty(5, 0, dtype=t, device="cuda"), m.out(5, 30)
    pg.gated(X5, Wn, Wn, en)
    pg.gated_backward(en, X5, Wn, Wn, en, en, dX=dX, dWg=torch.empty_like(Wn), dWu=torch.empty_like(Wn))
    torch.cuda.synchronize()
    assert bool((dX == 0).all())
    m.check_frames()


def block(pg, p, out, ws=None, stream=None):
    """A feed-forward block and its backward pass: H = silu(X Wg) * (X Wu), Y = H Wd + X."""
    k = dict(workspace=ws, stream=stream)
    pg.gated(p["X"], p["Wg"], p["Wu"], out["H"], act="silu", G=out["G"], U=out["U"], **k)
    pg.linear(out["H"], p["Wd"], out["Y"], bias=p["b"], residual=p["X"], **k)
    pg.linear_backward(p["dY"], out["H"], p["Wd"], dX=out["dH"], dW=out["dWd"], dbias=out["db"], **k)
    pg.gated_backward(out["dH"], p["X"], p["Wg"], p["Wu"], out["G"], out["U"], dX=out["dX"], dWg=out["dWg"],
                      dWu=out["dWu"], **k)


def block_state(M, D, F, t, seed, order="nk"):
    m = Maker(seed, t)
    p = dict(X=m.rows(M, D), Wg=m.weight(D, F, order), Wu=m.weight(D, F, order), Wd=m.weight(F, D, order),
             b=m.vector(D), dY=m.rows(M, D))

    def outs():
        n = Maker(0, t)
        return dict(H=n.out(M, F), G=n.out(M, F), U=n.out(M, F), Y=n.out(M, D), dH=n.out(M, F), dX=n.out(M, D),
                    dWd=n.weight_out(F, D, order), db=n.vector_out(D), dWg=n.weight_out(D, F, order),
                    dWu=n.weight_out(D, F, order))
    return p, outs


def same_bits(a, b):
    return all(torch.equal(a[k].contiguous().view(torch.uint8), b[k].contiguous().view(torch.uint8)) for k in a)


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("M,D,F", [(200, 96, 260), (1, 256, 520), (37, 200, 1032)])
def test_block_against_autograd(pg, M, D, F, order):
    """The four operators together in fp32 against autograd in 64 bits.  Each
    stage's inputs carry the error of the one before: products of K <= 1032 unit
    normals by weights of variance 1/K are off by at most K 2^-24 of their
    magnitudes; through four products the relative error of the whole (in the
    2-norm, where errors of either sign do not add up in full) stays
    below 4 * 1032 * 2^-24 = 2.5e-4."""
    say("block", (M, D, F), order)
    p, outs = block_state(M, D, F, torch.float32, M + F, order)
    o = outs()
    block(pg, p, o)
    torch.cuda.synchronize()
    q = {k: d64(v).requires_grad_() for k, v in p.items()}
    H = torch.nn.functional.silu(q["X"] @ q["Wg"]) * (q["X"] @ q["Wu"])
    Y = H @ q["Wd"] + q["b"] + q["X"]
    grads = torch.autograd.grad(Y, (q["X"], q["Wg"], q["Wu"], q["Wd"], q["b"]), q["dY"].detach())
    want = dict(zip(("dX", "dWg", "dWu", "dWd", "db"), grads), H=H, Y=Y)
    want["dX"] = want["dX"] - q["dY"]  # the skip connection's share is dY itself
    for k, w in want.items():
        w = w.detach()
        rel = float((d64(o[k]) - w).norm() / w.norm())
        assert rel < 2.5e-4, (k, rel)


@pytest.mark.parametrize("dtype", ["f32"])
def test_gradients_against_differences(pg, dtype):
    """sum(C * H) along a direction: the central difference over a step h of the
    library's own forward pass against the backward pass.  The difference is
    off by h^2 / 6 times the third derivative along the direction, and by the
    forward pass's error over h.  With directions of norm about sqrt(size) and
    weights of variance 1/K, changes of G and U per unit step are unit normals:
    |third derivative| per element is below 10 |C| (silu''' <= 0.5 times cubes of
    normals, and products with U's change), so over 24 x 40 elements of random
    sign 10 sqrt(960) = 310: with h = 2^-6 that is 310 h^2 / 6 = 0.013; the
    forward error 960 * 24 * 2^-24 / 2 h < 0.05 in the worst case."""
    say("differences")
    M, N, K, h = 24, 40, 16, 2.0 ** -6
    m = Maker(11, torch.float32)
    X, Wg, Wu, C = m.rows(M, K), m.weight(K, N, "kn"), m.weight(K, N, "nk").t().contiguous().t(), m.rows(M, N)
    Wu = Wu.contiguous()
    bg, bu = m.vector(N), m.vector(N)
    base = dict(X=X, Wg=Wg, Wu=Wu, bg=bg, bu=bu)
    H, G, U = (torch.empty(M, N, device="cuda") for _ in range(3))

    def value(s, way):
        a = {k: (v + s * way[k]).contiguous() if k in way else v for k, v in base.items()}
        pg.gated(a["X"], a["Wg"], a["Wu"], H, bias_g=a["bg"], bias_u=a["bu"], G=G, U=U)
        return float((H.double() * C.double()).sum())

    value(0.0, {})
    out = dict(X=torch.empty_like(X), Wg=torch.empty_like(Wg), Wu=torch.empty_like(Wu), bg=torch.empty_like(bg),
               bu=torch.empty_like(bu))
    pg.gated_backward(C, X, Wg, Wu, G, U, dX=out["X"], dWg=out["Wg"], dWu=out["Wu"], dbias_g=out["bg"],
                      dbias_u=out["bu"])
    for k, g in out.items():
        way = {k: (m.rows(*base[k].shape, K ** -0.5 if k[0] == "W" else 1.0) if base[k].dim() == 2 else m.vector(N))}
        slope = float((g.double() * way[k].double()).sum())
        diff = (value(h, way) - value(-h, way)) / (2 * h)
        assert abs(diff - slope) < 0.07, (k, diff, slope)


def test_graph_replays_equal_the_eager_call(pg):
    say("graph")
    p, outs = block_state(300, 256, 520, torch.bfloat16, 5)
    eager, o = outs(), outs()
    block(pg, p, eager)
    block(pg, p, o)
    torch.cuda.synchronize()
    assert same_bits(eager, o)  # the same call twice
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block(pg, p, o)
    x = torch.ones(1 << 20, device="cuda")
    for rep in range(4):
        for v in o.values():
            v.fill_(SENTINEL)
        x.mul_(1.5).add_(rep)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same_bits(eager, o), rep


def test_two_graphs_share_a_workspace(pg):
    """Replayed one after the other on one stream; the workspace holds nothing between them."""
    say("two graphs")
    need = max(pg.pgemm_gated_backward_workspace(300, 520, 256, 2),
               pg.pgemm_linear_backward_workspace(300, 256, 520, 0, 2),
               pg.pgemm_gated_workspace(300, 520, 256, 2),
               pg.pgemm_linear_workspace(300, 256, 520, 2),
               pg.pgemm_gated_backward_workspace(70, 520, 256, 2),
               pg.pgemm_linear_backward_workspace(70, 256, 520, 0, 2),
               pg.pgemm_gated_workspace(70, 520, 256, 2),
               pg.pgemm_linear_workspace(70, 256, 520, 2))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    runs = []
    for M in (300, 70):
        p, outs = block_state(M, 256, 520, torch.bfloat16, M)
        eager, o = outs(), outs()
        block(pg, p, eager)
        block(pg, p, o, ws)
        torch.cuda.synchronize()
        assert same_bits(eager, o)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            block(pg, p, o, ws)
        runs.append((g, eager, o, p))  # the graph reads p: it has to live as long
    for rep in range(3):
        for g, eager, o, _ in runs + runs[::-1]:
            for v in o.values():
                v.fill_(SENTINEL)
            g.replay()
            torch.cuda.synchronize()
            assert same_bits(eager, o), rep
            ws.fill_(rep)


def test_other_streams(pg):
    """Two blocks on two streams at once, each with its own workspace, by stream object and by handle."""
    say("streams")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for s, M in ((a, 190), (b, 260)):
        p, outs = block_state(M, 512, 1032, torch.float16, M)
        eager, o = outs(), outs()
        block(pg, p, eager)
        runs.append((s, p, eager, o))
    torch.cuda.synchronize()
    for rep in range(5):
        for i, (s, p, eager, o) in enumerate(runs):
            s.wait_stream(torch.cuda.current_stream())
            block(pg, p, o, stream=s if rep % 2 else s.cuda_stream)
        torch.cuda.synchronize()
        for s, p, eager, o in runs:
            assert same_bits(eager, o), rep
            for v in o.values():
                v.fill_(SENTINEL)
        torch.cuda.synchronize()


def test_residual_in_place_and_shared_weight_buffers(pg):
    say("in place")
    t = torch.bfloat16
    m = Maker(21, t)
    X, W, Y = m.rows(70, 200), m.weight(200, 96, "nk"), m.rows(70, 96)
    start = Y.clone()
    pg.linear(X, W, Y, residual=Y, act="gelu")
    ref.check("Y", Y, ref.linear(X, W, None, start, "gelu", t)[0])
    # Wg and Wu as halves of one parameter, G and U as halves of one buffer
    for order in ("kn", "nk"):
        W2 = m.weight(200, 2 * 96, order)
        GU, H = m.out(70, 2 * 96), m.out(70, 96)
        pg.gated(X, W2[:, :96], W2[:, 96:], H, G=GU[:, :96], U=GU[:, 96:])
        h, g, u = ref.gated(X, W2[:, :96], W2[:, 96:], None, None, "silu", t)
        for name, got, want in (("H", H, h), ("G", GU[:, :96], g), ("U", GU[:, 96:], u)):
            ref.check(name, got, want)


def test_long_leading_dimensions(pg):
    """Rows a million elements apart: offsets beyond 2^31 bytes from the base."""
    say("long rows")
    t = torch.bfloat16
    ld, M, N, K = (1 << 20) + 8, 1500, 72, 130
    big = torch.zeros(M * ld, dtype=t, device="cuda").view(M, ld)
    m = Maker(31, t)
    X = big[:, :K]
    X.copy_(m.rows(M, K))
    W, Y = m.weight(K, N, "nk"), big[:, K + 6:K + 6 + N]
    pg.linear(X, W, Y, act="relu")
    ref.check("Y", Y, ref.linear(X, W, None, None, "relu", t)[0])
    dY, dX = big[:, 300:300 + N], big[:, 400:400 + K]
    dY.copy_(m.rows(M, N))
    dW, db = m.weight_out(K, N, "nk"), m.vector_out(N)
    pg.linear_backward(dY, X, W, Z=Y, act="gelu", dX=dX, dW=dW, dbias=db)
    for name, got, want in zip(("dX", "dW", "db"), (dX, dW, db), ref.linear_backward(dY, X, W, Y, "gelu", t)):
        ref.check(name, got, want)


def test_offsets_beyond_32_bits(pg):
    """Outputs and weights of more than 2^31 elements: small integers, so every sum is exact."""
    big, other, step, t = 70000, 33000, 5000, torch.bfloat16

    def whole(*shape):
        return torch.randint(-2, 3, shape, dtype=torch.int8, device="cuda").to(t)

    # a large output: Y[big][other], and dW in the other direction
    X, W = whole(big, 16), whole(16, other)
    Y = torch.full((big, other), SENTINEL, dtype=torch.float32, device="cuda")
    say("large output")
    pg.linear(X, W, Y)
    for r in range(0, big, step):
        assert torch.equal(Y[r:r + step].double(), X[r:r + step].double() @ W.double()), r
    dW, A = Y.fill_(SENTINEL), X.t().contiguous()  # dW = A^T dY
    say("large weight gradient")
    pg.linear_backward(W, A, torch.empty(big, other, dtype=t, device="cuda"), dW=dW)
    for r in range(0, big, step):
        assert torch.equal(dW[r:r + step].double(), X[r:r + step].double() @ W.double()), r
    del Y, dW

    # a large weight, each storage order, forward (few rows) and as operand of dX
    B = whole(big, other)
    for M in (2, 200):
        x, dy = whole(M, other), whole(M, big)
        y, dx = torch.empty(M, big, dtype=torch.float32, device="cuda"), torch.empty(M, other, dtype=t, device="cuda")
        want = torch.cat([x.double() @ B[r:r + step].double().t() for r in range(0, big, step)], 1)
        say("large weight", M)
        pg.linear(x, B.t(), y)  # W[N][K]
        assert torch.equal(y.double(), want)
        wantx = sum(dy[:, r:r + step].double() @ B[r:r + step].double() for r in range(0, big, step))
        pg.linear_backward(dy, x, B.t(), dX=dx)
        assert torch.equal(dx, wantx.float().to(t))
        y2, dx2 = torch.empty(M, other, dtype=torch.float32, device="cuda"), torch.empty(M, big, dtype=t, device="cuda")
        pg.linear(dy, B, y2)  # W[K][N]
        assert torch.equal(y2.double(), wantx)
        pg.linear_backward(x, dy, B, dX=dx2)
        assert torch.equal(dx2, want.float().to(t))
