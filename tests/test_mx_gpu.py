"""The norm and the microscaled operators on the GPU against plain 64-bit forms."""
import pytest
import torch

import mx_reference as ref
from software_pipelined_tiled_loop_amd import binding as pg

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(g, r, c, dtype, pad=0, scale=1.0, fill=None):
    """r x c values `pad` elements apart; fill: an output, with what lies between the rows told apart."""
    if fill is not None:
        return torch.full((r, c + pad), fill, dtype=dtype, device="cuda")[:, :c]
    return torch.randn(r, c + pad, generator=g, device="cuda").mul_(scale).to(dtype)[:, :c]


def between(t, c):
    """The elements behind the columns of a padded output."""
    return t.as_strided((t.shape[0], max(t.stride(0) - c, 0)), (t.stride(0), 1), t.storage_offset() + c)[:-1]


NORMS = [(1, 8), (1, 1), (3, 7), (2, 513), (5, 512), (4, 1024), (3, 1025), (33, 2048), (2, 2049), (1, 4096), (7, 4001),
         (2, 8192), (3, 8200), (2, 16384), (2, 16391), (1, 40000), (700, 96), (0, 64), (5, 32)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N", NORMS)
def test_norm(M, N, dtype):
    t, g = TYPES[dtype], gen(M * 100003 + N)
    pad = N % 3
    X, R, w = rows(g, M, N, t, pad), rows(g, M, N, t, 0, 2.0), torch.randn(N, generator=g, device="cuda").to(t)
    for residual, weight, out in ((None, w, t), (R, w, torch.float32), (R, None, t)):
        Y, H = rows(None, M, N, out, pad, fill=9.0), rows(None, M, N, t, pad, fill=9.0)
        mx = [pg.mx_empty(M, N, f, "cuda") for f in ("mx8", "mx4")]
        assert pg.rms_norm(X, weight, Y, residual=residual, H=H, mx=mx[0], eps=EPS) is Y
        assert pg.rms_norm(X, weight, residual=residual, mx=mx[1], eps=EPS) is mx[1]
        torch.cuda.synchronize()
        (h, eh), (y, ey) = ref.norm(X, residual, weight, EPS)
        ref.close(H, ref.round_out(h, eh, t), "H")
        ref.close(Y, ref.round_out(y, ey, out), "Y")
        for m in mx:
            ref.check_blocks(m, y, ey, ref.form_of(m))
        if M and pad:
            assert bool((between(Y, N) == 9).all()) and bool((between(H, N) == 9).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,N", NORMS)
def test_norm_backward(M, N, dtype):
    t, g = TYPES[dtype], gen(M * 100019 + N)
    pad = N % 4
    H, dY, dH = rows(g, M, N, t, pad, 2.0), rows(g, M, N, t), rows(g, M, N, t, 1)
    w = torch.randn(N, generator=g, device="cuda").to(t)
    for weight, dh, gt in ((w, None, t), (w, dH, torch.float32), (None, dH, t)):
        dX, dw = rows(None, M, N, t, pad, fill=9.0), torch.full((N,), 9.0, dtype=gt, device="cuda")
        got = pg.rms_norm_backward(dY, H, weight, dH=dh, dX=dX, dweight=dw, eps=EPS)
        assert got[0] is dX and got[1] is dw
        torch.cuda.synchronize()
        (dx, edx), (dwv, edw) = ref.norm_backward(dY, H, weight, dh, EPS)
        ref.close(dX, ref.round_out(dx, edx, t), "dX")
        ref.close(dw, ref.round_out(dwv, edw, gt), "dweight")
        if M and pad:
            assert bool((between(dX, N) == 9).all())
        alone = torch.empty_like(dX)
        pg.rms_norm_backward(dY, H, weight, dH=dh, dX=alone, eps=EPS)
        assert torch.equal(alone, dX)


def special(dtype, rows_, K, seed):
    """Values over the type's range, ties of both formats, zeros, infinities and NaN in single blocks."""
    g = gen(seed)
    t = TYPES[dtype]
    x = torch.randn(rows_, K, generator=g, device="cuda")
    span = 40 if dtype == "f16" else 200
    e = torch.randint(-span // 2, span // 3 if dtype != "f16" else 12, (rows_, -(-K // 32)), generator=g, device="cuda")
    x = x * torch.ldexp(torch.ones_like(e, dtype=torch.float32), e).repeat_interleave(32, 1)[:, :K]
    if rows_ > 4 and K >= 64:
        ties = torch.arange(32, device="cuda") * 0.25  # every tie of e2m1 up to 7.75
        x[0, :32] = ties
        x[1, :32] = -ties.clamp_max(6.999)
        x[2, :32] = torch.arange(32, device="cuda") * 16 + 8  # up to 504: ties of the largest binade
        x[2, 29:32] = 1.0  # the largest entry is 456: it rounds to 448
        x[3, :32] = 0.0
        x[3, 0] = -0.0
        x[4, 5] = float("inf")
        x[4, 40] = float("nan")
    return x.to(t)


@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,K", [(1, 1), (1, 4096), (5, 31), (3, 33), (6, 255), (7, 256), (70, 257), (33, 4001), (129, 96),
                                 (64, 1000)])
def test_quantize(R, K, dtype, form):
    x = special(dtype, R, K, R * 7919 + K)
    want = ref.quantize(x, form)
    wide = torch.zeros(R, K + 3, dtype=x.dtype, device="cuda")
    wide[:, :K] = x
    turned = torch.zeros(K, R + 5, dtype=x.dtype, device="cuda")
    turned[:, :R] = x.t()
    for X in (x, wide[:, :K], x.t().contiguous().t(), turned[:, :R].t()):
        Q, S = pg.mx_empty(R, K, form, "cuda")
        Q.fill_(0xEE), S.fill_(0xEE)
        assert pg.mx_quantize(X, (Q, S))[0] is Q
        assert torch.equal(Q.cpu(), want[0]) and torch.equal(S.cpu(), want[1])
    for out in TYPES.values():
        V = torch.full((R, K + 2), 9.0, dtype=out, device="cuda")
        assert pg.mx_dequantize((Q, S), V[:, :K]) is not None
        v = ref.values(Q, S, form)[:, :K]
        assert torch.equal(V[:, :K].cpu().nan_to_num(-1.25), v.to(out).nan_to_num(-1.25)), out
        assert bool((V[:, K:] == 9).all())


def test_blocks_of_other_strides_and_types():
    """Codes and scales as slices of wider tensors and in torch's 8-bit float types; what lies between stays."""
    x = torch.randn(40, 500, device="cuda").bfloat16()
    want = ref.quantize(x, "mx8")
    Q, S = torch.full((40, 528), 7, dtype=torch.uint8, device="cuda"), torch.full((40, 20), 7, dtype=torch.uint8, device="cuda")
    pg.mx_quantize(x, (Q[:, :512].view(torch.float8_e4m3fn), S[:, :16].view(torch.float8_e8m0fnu)))
    assert torch.equal(Q[:, :512].cpu(), want[0]) and torch.equal(S[:, :16].cpu(), want[1])
    assert bool((Q[:, 512:] == 7).all()) and bool((S[:, 16:] == 7).all())


def weights(g, N, K, scale=1.0):
    return pg.mx_quantize(torch.randn(N, K, generator=g, device="cuda").mul_(scale), pg.mx_empty(N, K, "mx4", "cuda"))


PRODUCTS = [(1, 1, 1), (1, 16, 256), (1, 130, 300), (7, 33, 64), (16, 64, 512), (17, 40, 700), (33, 200, 1000), (48, 77, 4001),
            (64, 64, 1024), (65, 130, 513), (130, 260, 256), (257, 300, 2000), (300, 515, 130), (0, 5, 64), (5, 0, 64)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_linear(M, N, K, form, dtype):
    t, g = TYPES[dtype], gen(M * 31 + N * 7 + K)
    X = pg.mx_quantize(torch.randn(M, K, generator=g, device="cuda"), pg.mx_empty(M, K, form, "cuda"))
    W = weights(g, N, K, K ** -0.5)
    for act, bias, residual in (("none", False, False), ("silu", True, True), ("relu", True, False), ("gelu", False, True),
                                ("gelu_tanh", True, True)):
        b = torch.randn(N, generator=g, device="cuda").to(t) if bias else None
        R = rows(g, M, N, t, 3) if residual else None
        Y = rows(None, M, N, t, 1, fill=9.0)
        assert pg.mx_linear(X, W, Y, bias=b, residual=R, act=act) is Y
        ref.close(Y, ref.linear(X, W, b, R, act, t), act)
        if M:
            assert bool((between(Y, N) == 9).all())
        if residual:  # the residual may be the output itself
            again = R.clone()
            pg.mx_linear(X, W, again, bias=b, residual=again, act=act)
            assert torch.equal(again, Y)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("form", ["mx8", "mx4"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_gated(M, N, K, form, dtype):
    t, g = TYPES[dtype], gen(M * 37 + N * 11 + K)
    X = pg.mx_quantize(torch.randn(M, K, generator=g, device="cuda"), pg.mx_empty(M, K, form, "cuda"))
    Wg, Wu = weights(g, N, K, K ** -0.5), weights(g, N, K, K ** -0.5)
    for act, bias in (("silu", False), ("gelu_tanh", True), ("relu", True)):
        bg, bu = (torch.randn(N, generator=g, device="cuda").to(t) if bias else None for _ in range(2))
        H = rows(None, M, N, t, 5, fill=9.0)
        assert pg.mx_gated(X, Wg, Wu, H, bias_g=bg, bias_u=bu, act=act) is H
        ref.close(H, ref.gated(X, Wg, Wu, bg, bu, act, t), act)
        if M:
            assert bool((between(H, N) == 9).all())


def test_products_of_nothing():
    """No entries: bias, activation and residual alone."""
    X, W = pg.mx_empty(3, 0, "mx8", "cuda"), pg.mx_empty(5, 0, "mx4", "cuda")
    b, R = torch.randn(5, device="cuda"), torch.randn(3, 5, device="cuda")
    Y = pg.mx_linear(X, W, torch.empty(3, 5, device="cuda"), bias=b, residual=R, act="relu")
    assert torch.equal(Y, b.clamp_min(0) + R)
