"""Every compiled kernel of the feed-forward operators with all of its options: sizes
from linear_shapes.py (test_linear_plans.py holds that the planner takes every tile
class there, whole and split, and every few-rows kernel), ragged in each direction,
with biases, activations, kept pre-activations, and the residual in Y itself.  Frames
and bounds as in test_linear_gpu.py and linear_reference.py."""
import pytest
import torch

import linear_reference as ref
import linear_shapes
from test_linear_gpu import TYPES, Maker, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pg():
    from software_pipelined_tiled_loop_amd import binding
    return binding


@pytest.fixture(autouse=True)
def on_gpu(monkeypatch):
    """The 64-bit form evaluated on the GPU (float64 products), for the large sizes."""
    monkeypatch.setattr(ref, "WHERE", "cuda")


def forward(pg, m, kind, M, N, K, t, i):
    order, act = ("kn", "nk")[kind & 1], ref.ACTS[i % 5]
    wide = torch.float32 if i % 4 == 3 else t  # Y and the residual
    X, W = m.rows(M, K), m.weight(K, N, order)
    b = m.vector(N) if i % 3 else None
    Z = m.out(M, N) if i % 2 else None
    Y = m.out(M, N, wide)
    if kind < 2:
        R = m.rows(M, N, dtype=wide) if i % 5 else None
        if R is not None and i % 5 != 1:  # in place
            Y.copy_(R)
        pg.linear(X, W, Y, bias=b, residual=None if R is None else Y if i % 5 != 1 else R, act=act, Z=Z)
        y, z = ref.linear(X, W, b, R, act, wide)
        return [("Y", Y, y), ("Z", Z, z)]
    Wu, bu, U = m.weight(K, N, order), m.vector(N) if i % 2 else None, m.out(M, N) if i % 3 != 1 else None
    pg.gated(X, W, Wu, Y, bias_g=b, bias_u=bu, act=act, G=Z, U=U)
    h, g, u = ref.gated(X, W, Wu, b, bu, act, wide)
    return [("H", Y, h), ("G", Z, g), ("U", U, u)]


def backward(pg, m, kind, M, N, K, t, i):
    """dX or dW alone, of the one or the other operator."""
    order, gated = ("kn", "nk")[kind & 1], (kind >> 1) & 1
    act, wide = ref.ACTS[i % 5], torch.float32 if i % 4 == 3 else t
    dY, X, Z = m.rows(M, N), m.rows(M, K), m.rows(M, N)
    W = m.weight(K, N, order)
    dX = m.out(M, K) if kind < 8 else None
    dW = m.weight_out(K, N, order, wide) if kind >= 8 else None
    if not gated:
        pg.linear_backward(dY, X, W, Z=Z, act=act, dX=dX, dW=dW)
        dx, dw, _ = ref.linear_backward(dY, X, W, Z, act, wide)
        return [("dX", dX, dx), ("dW", dW, dw)]
    U, Wu = m.rows(M, N), m.weight(K, N, order)
    dWu = m.weight_out(K, N, order, wide) if kind >= 8 else None
    pg.gated_backward(dY, X, W, Wu, Z, U, act=act, dX=dX, dWg=dW, dWu=dWu)
    dx, dw, dwu, _, _ = ref.gated_backward(dY, X, W, Wu, Z, U, act, wide)
    return [("dX", dX, dx), ("dWg", dW, dw), ("dWu", dWu, dwu)]


def run(pg, dtype, i, kind, M, N, K):
    say("kernel", dtype, kind, (M, N, K), i)
    t = TYPES[dtype]
    m = Maker(900 + i, t, (0, 1, 8, 3)[i % 4], (0, 1, 3)[i % 3])
    i += list(TYPES).index(dtype)  # the options walk with the type too
    for name, got, want in (forward if kind < 4 else backward)(pg, m, kind, M, N, K, t, i):
        if got is not None:
            ref.check(name, got, want)
    m.check_frames()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("i", range(len(linear_shapes.TILES)))
def test_tiles(pg, dtype, i):
    run(pg, dtype, i, *linear_shapes.TILES[i])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("i", range(len(linear_shapes.FEW)))
def test_few_rows(pg, dtype, i):
    run(pg, dtype, i, *linear_shapes.FEW[i])


@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_residual_in_place_over_several_tiles_and_a_join(pg, dtype, order):
    """R = Y where the epilogue reads ahead (whole tiles of 256 x 256), and through the join."""
    kind, t = ("kn", "nk").index(order), TYPES[dtype]
    for M, N, K in [s[1:] for s in linear_shapes.TILES if s[0] == kind]:
        say("in place", dtype, order, (M, N, K))
        m = Maker(M, t, 1, 1)
        X, W, R, Y = m.rows(M, K), m.weight(K, N, order), m.rows(M, N), m.out(M, N)
        Y.copy_(R)
        pg.linear(X, W, Y, residual=Y, act="silu")
        ref.check("Y", Y, ref.linear(X, W, None, R, "silu", t)[0])
        m.check_frames()
