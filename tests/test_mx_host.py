"""Host checks of the norm and of the microscaled operators (no GPU): refusals of the C
entry points and of the torch wrappers before anything is launched, and workspaces."""
import os
import re

import pytest
import torch

import mx_reference as ref
from software_pipelined_tiled_loop_amd import binding as lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # never dereferenced: every call below is refused first
OK, INVALID, DTYPE, LARGE = 0, -1, -2, -7


def call(function, defaults):
    def f(**k):
        assert set(k) <= set(defaults)
        return function(*dict(defaults, **k).values(), None)
    return f


norm = call(lib.pgemm_rms_norm, dict(M=6, N=300, X=FAKE, ldx=300, R=FAKE, ldr=300, w=FAKE, eps=1e-6, H=FAKE, ldh=300, Y=FAKE,
                                     ldy=300, out=2, Q=FAKE, ldq=512, S=FAKE, lds=16, form=0, dtype=2))
norm_grad = call(lib.pgemm_rms_norm_backward, dict(M=600, N=300, dY=FAKE, lddy=300, H=FAKE, ldh=300, w=FAKE, eps=1e-6, dH=FAKE,
                                                   lddh=300, dX=FAKE, lddx=300, dw=FAKE, grad=2, dtype=2, ws=FAKE, n=1 << 40))
quantize = call(lib.pgemm_mx_quantize, dict(M=6, K=300, X=FAKE, ldx=300, order=1, dtype=2, Q=FAKE, ldq=512, S=FAKE, lds=16,
                                            form=0))
dequantize = call(lib.pgemm_mx_dequantize, dict(M=6, K=300, Q=FAKE, ldq=512, S=FAKE, lds=16, form=0, X=FAKE, ldx=300, dtype=2))
linear = call(lib.pgemm_mx_linear, dict(M=6, N=40, K=300, XQ=FAKE, ldxq=512, XS=FAKE, ldxs=16, form=0, WQ=FAKE, ldwq=256,
                                        WS=FAKE, ldws=16, b=FAKE, R=FAKE, ldr=40, act=1, Y=FAKE, ldy=40, dtype=2, ws=None,
                                        n=0))
gated = call(lib.pgemm_mx_gated, dict(M=6, N=40, K=300, XQ=FAKE, ldxq=512, XS=FAKE, ldxs=16, form=0, WgQ=FAKE, WuQ=FAKE,
                                      ldwq=256, WgS=FAKE, WuS=FAKE, ldws=16, bg=FAKE, bu=FAKE, act=2, H=FAKE, ldh=40, dtype=2,
                                      ws=None, n=0))

COMMON = [(dict(dtype=3), DTYPE), (dict(dtype=9), DTYPE), (dict(M=-1), INVALID), (dict(M=1 << 31), LARGE)]
BLOCKS = [(dict(Q=FAKE + 8), INVALID), (dict(S=FAKE + 2), INVALID), (dict(ldq=511), INVALID), (dict(ldq=256), INVALID),
          (dict(ldq=520), INVALID), (dict(lds=8), INVALID), (dict(lds=17), INVALID), (dict(form=2), INVALID),
          (dict(form=-1), INVALID), (dict(ldq=1 << 21), LARGE), (dict(S=None), INVALID)]
NORM = COMMON + [(dict(N=-1), INVALID), (dict(N=1 << 21), LARGE), (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID),
                 (dict(eps=float("inf")), INVALID), (dict(w=FAKE + 1), INVALID), (dict(ldh=299), INVALID)]
PRODUCT = COMMON + [(dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(K=1 << 21), LARGE), (dict(act=5), INVALID),
                    (dict(act=-1), INVALID), (dict(form=2), INVALID), (dict(XQ=None), INVALID), (dict(XS=None), INVALID),
                    (dict(XQ=FAKE + 4), INVALID), (dict(XS=FAKE + 1), INVALID), (dict(ldxq=256), INVALID),
                    (dict(ldxq=520), INVALID), (dict(ldxs=8), INVALID), (dict(ldxs=18), INVALID), (dict(ldwq=128), INVALID),
                    (dict(ldwq=264), INVALID), (dict(ldws=12), INVALID), (dict(ldwq=1 << 21), LARGE), (dict(ldws=1 << 21), LARGE),
                    (dict(M=1 << 28, N=1 << 20), LARGE)]


@pytest.mark.parametrize("f,args,code", [(norm, *c) for c in NORM + BLOCKS + [
    (dict(X=None), INVALID), (dict(X=FAKE + 1), INVALID), (dict(ldx=299), INVALID), (dict(ldr=12), INVALID), (dict(out=1), INVALID),
    (dict(ldy=299), INVALID), (dict(Y=FAKE + 2, out=0), INVALID), (dict(Q=None), INVALID), (dict(ldx=1 << 21), LARGE)]]
    + [(norm_grad, *c) for c in NORM + [
        (dict(dY=None), INVALID), (dict(H=None), INVALID), (dict(lddy=299), INVALID), (dict(lddh=299), INVALID),
        (dict(lddx=299), INVALID), (dict(grad=1), INVALID), (dict(dw=FAKE + 2, grad=0), INVALID), (dict(ws=None), INVALID),
        (dict(ws=FAKE + 8), INVALID), (dict(n=16), INVALID)]]
    + [(quantize, *c) for c in COMMON + BLOCKS + [
        (dict(K=-1), INVALID), (dict(order=2), INVALID), (dict(ldx=299), INVALID), (dict(order=0, ldx=5), INVALID),
        (dict(X=None), INVALID), (dict(X=FAKE + 1), INVALID), (dict(Q=None), INVALID), (dict(K=1 << 21), INVALID)]]
    + [(dequantize, *c) for c in COMMON + BLOCKS + [
        (dict(K=-1), INVALID), (dict(ldx=299), INVALID), (dict(X=None), INVALID), (dict(Q=None), INVALID), (dict(K=1 << 21), LARGE)]]
    + [(linear, *c) for c in PRODUCT + [
        (dict(WQ=None), INVALID), (dict(WS=None), INVALID), (dict(b=FAKE + 1), INVALID), (dict(ldr=39), INVALID),
        (dict(Y=None), INVALID), (dict(ldy=39), INVALID), (dict(Y=FAKE + 1), INVALID)]]
    + [(gated, *c) for c in PRODUCT + [
        (dict(WgQ=None), INVALID), (dict(WuQ=None), INVALID), (dict(WgS=None), INVALID), (dict(WuS=FAKE + 3), INVALID),
        (dict(bu=FAKE + 1), INVALID), (dict(H=None), INVALID), (dict(ldh=39), INVALID)]])
def test_refused_by_the_c_entry(f, args, code):
    assert f(**args) == code, lib.pgemm_strerror(f(**args))


def test_empty_calls_launch_nothing():
    assert norm(M=0, X=None, R=None, H=None, Y=None, Q=None, S=None) == OK
    assert norm(N=0, X=None, R=None, H=None, Y=None, Q=None, S=None) == OK
    assert norm(H=None, Y=None, Q=None, S=None) == OK  # nothing is asked for
    assert norm_grad(N=0, dY=None, H=None, dH=None, dX=None) == OK
    assert norm_grad(M=0, dY=None, H=None, dX=FAKE, dw=None, ws=None, n=0) == OK
    assert quantize(M=0, X=None, Q=None, S=None) == OK and dequantize(K=0, X=None, Q=None, S=None) == OK
    assert linear(M=0, XQ=None, XS=None, WQ=None, WS=None, R=None, Y=None) == OK
    assert gated(N=0, XQ=None, XS=None, WgQ=None, WuQ=None, WgS=None, WuS=None, H=None) == OK


def test_workspaces():
    assert lib.pgemm_rms_norm_backward_workspace(0, 64, 2) == 0
    assert lib.pgemm_rms_norm_backward_workspace(1, 64, 2) == 0  # few rows: no sums to join
    assert lib.pgemm_rms_norm_backward_workspace(1, 1 << 20, 2) == 4 << 20  # a row too long for the registers keeps them there
    assert lib.pgemm_rms_norm_backward_workspace(4096, 4096, 2) % 16384 == 0
    assert lib.pgemm_rms_norm_backward_workspace(5, 4, 3) == DTYPE
    for f in (lib.pgemm_mx_linear_workspace, lib.pgemm_mx_gated_workspace):
        assert f(1, 1, 1, 0, 2) >= 0 and f(1, 1, 1, 2, 2) == INVALID and f(-1, 1, 1, 0, 2) == INVALID
        assert f(1, 1 << 21, 1, 1, 2) == LARGE and f(1, 1, 1, 0, 3) == DTYPE
        assert f(300, (1 << 21) - 1, 1, 0, 0) == LARGE and f(300, (1 << 21) - 8, 1, 0, 0) > 0
        # fp32 outputs of many MX8 rows keep the values of both operands
        assert f(4096, 4096, 4096, 0, 0) >= 2 * 4096 * 4096 * 2 and f(4096, 4096, 4096, 1, 0) < 1 << 20


def test_every_declared_function_is_bound():
    with open(os.path.join(ROOT, "include", "pgemm.h")) as f:
        names = set(re.findall(r"^\w+ (pgemm_(?:rms|mx)_\w*)\(", f.read(), re.M))
    assert len(names) == 9 and names <= set(lib.EXPORTED)
    for name in names:
        assert getattr(lib, name) is not None and getattr(lib._lib, name).argtypes


# ---- the torch wrappers ----------------------------------------------------------------------


def host(M=6, N=40, K=300, form="mx8", t=torch.bfloat16):
    e = lambda *s: torch.zeros(*s, dtype=t)  # noqa: E731
    return dict(X=lib.mx_empty(M, K, form, "cpu"), W=lib.mx_empty(N, K, "mx4", "cpu"), Y=e(M, N), b=e(N), R=e(M, N))


def refused(match, f, *a, **k):
    with pytest.raises(ValueError, match=match):
        f(*a, **k)


def test_norm_wrappers_refuse():
    x = torch.zeros(6, 300).bfloat16()
    y, w = torch.empty_like(x), torch.zeros(300).bfloat16()
    refused("on a GPU", lib.rms_norm, x, w, y)
    refused("one of Y, H and mx", lib.rms_norm, x, w)
    refused("unsupported dtype", lib.rms_norm, x.double(), None, y.double())
    refused("weight must be a contiguous vector", lib.rms_norm, x, w[:5], y)
    refused("weight must be torch.bfloat16", lib.rms_norm, x, w.float(), y)
    refused("Y is", lib.rms_norm, x, w, y[:, :4])
    refused("residual must be torch.bfloat16", lib.rms_norm, x, w, y, residual=x.float())
    refused("row-major", lib.rms_norm, x.t().contiguous().t(), w, y)
    refused("row-major", lib.rms_norm, x, w, y, residual=x[:1].expand(6, 300))
    refused("X and Y overlap", lib.rms_norm, x, w, x)
    refused("on a GPU", lib.rms_norm, x, w, y, residual=x, H=x)  # in place is served
    refused("on a GPU", lib.rms_norm, x, w, y, residual=y.clone(), H=x)
    refused("Y and H overlap", lib.rms_norm, x, w, y, H=y)
    refused("eps", lib.rms_norm, x, w, y, eps=-1)
    refused("eps", lib.rms_norm, x, w, y, eps=float("nan"))
    refused("eps", lib.rms_norm, x, w, y, eps="a")
    refused("pair", lib.rms_norm, x, w, y, mx=x)
    refused("pair", lib.rms_norm, x, w, y, mx=(x,))
    refused("rows of 256 entries, the call needs 512", lib.rms_norm, x, w, y, mx=lib.mx_empty(6, 256, "mx8", "cpu"))
    refused("needs 6 rows", lib.rms_norm, x, w, y, mx=lib.mx_empty(5, 300, "mx8", "cpu"))
    refused("on a GPU", lib.rms_norm, x, w, y, mx=lib.mx_empty(6, 300, "mx8", "cpu"))
    refused("matrix is needed", lib.rms_norm, w, None, w)
    refused("X is needed", lib.rms_norm, None, w, y)
    refused("on a GPU", lib.rms_norm_backward, y, x, w, dX=y.clone(), dweight=w.float())
    refused("dY is needed", lib.rms_norm_backward, None, x, w, dX=y)
    refused("dY and dX overlap", lib.rms_norm_backward, y, x, w, dX=y)
    refused("on a GPU", lib.rms_norm_backward, y, x, w, dH=y.clone(), dX=torch.empty_like(y))
    d = torch.empty_like(y)
    refused("on a GPU", lib.rms_norm_backward, y, x, w, dH=d, dX=d)
    refused("weight and dweight overlap", lib.rms_norm_backward, y, x, w, dweight=w)
    refused("dweight must be", lib.rms_norm_backward, y, x, w, dweight=w.half())


def test_mx_wrappers_refuse():
    x = torch.zeros(6, 300)
    refused("unknown format", lib.mx_empty, 1, 1, "mx6", "cpu")
    refused("not negative", lib.mx_empty, -1, 1, "mx4", "cpu")
    Q, S = lib.mx_empty(6, 300, "mx4", "cpu")
    assert Q.shape == (6, 256) and S.shape == (6, 16) and lib.mx_empty(2, 257, "mx8", "cpu")[0].shape == (2, 512)
    refused("X has unsupported", lib.mx_quantize, x.int(), (Q, S))
    refused("on a GPU", lib.mx_quantize, x, (Q, S))
    refused("on a GPU", lib.mx_quantize, torch.zeros(300, 6).t(), (Q, S))
    refused("unit stride along one axis", lib.mx_quantize, torch.zeros(6, 600)[:, ::2], (Q, S))
    refused("codes must be", lib.mx_quantize, x, (Q.int(), S))
    refused("scales must be", lib.mx_quantize, x, (Q, S.int()))
    refused("whole groups", lib.mx_quantize, x, (Q[:, :200], S))
    refused("whole groups", lib.mx_quantize, x, (Q, S[:, :12]))
    refused("rows a multiple of 16", lib.mx_quantize, x, (torch.zeros(6, 264, dtype=torch.uint8)[:, :256], S))
    refused("rows a multiple of 4", lib.mx_quantize, x, (Q, torch.zeros(6, 18, dtype=torch.uint8)[:, :16]))
    refused("mx and mx overlap", lib.mx_quantize, x, (Q, Q.view(-1)[:96].view(6, 16)))
    refused("pair", lib.mx_quantize, x, None)
    refused("entries, the call needs", lib.mx_dequantize, (Q, S), torch.zeros(6, 700))
    refused("on a GPU", lib.mx_dequantize, (Q, S), torch.zeros(6, 257))
    refused("needs 5 rows", lib.mx_dequantize, (Q, S), x[:5])
    refused("row-major", lib.mx_dequantize, (Q, S), torch.zeros(300, 6).t())
    h = host()
    refused("on a GPU", lib.mx_linear, h["X"], h["W"], h["Y"], bias=h["b"], residual=h["Y"])
    refused("unknown activation", lib.mx_linear, h["X"], h["W"], h["Y"], act="tanh")
    refused("unknown activation", lib.mx_linear, h["X"], h["W"], h["Y"], act=["relu"])
    refused("4-bit", lib.mx_linear, h["X"], lib.mx_empty(40, 300, "mx8", "cpu"), h["Y"])
    refused("entries, the call needs 512", lib.mx_linear, h["X"], lib.mx_empty(40, 200, "mx4", "cpu"), h["Y"])
    refused("needs 40 rows", lib.mx_linear, h["X"], lib.mx_empty(41, 300, "mx4", "cpu"), h["Y"])
    refused("needs 6 rows", lib.mx_linear, lib.mx_empty(7, 300, "mx4", "cpu"), h["W"], h["Y"])
    refused("bias must be torch.bfloat16", lib.mx_linear, h["X"], h["W"], h["Y"], bias=h["b"].float())
    refused("residual is", lib.mx_linear, h["X"], h["W"], h["Y"], residual=h["R"][:3])
    refused("Y has unsupported", lib.mx_linear, h["X"], h["W"], h["Y"].double())
    refused("pair", lib.mx_linear, h["Y"], h["W"], h["Y"])
    refused("on a GPU", lib.mx_gated, h["X"], h["W"], h["W"], h["Y"])
    wide = torch.zeros(40, 512, dtype=torch.uint8)[:, :256]
    refused("same strides", lib.mx_gated, h["X"], h["W"], (wide, h["W"][1]), h["Y"])
    refused("4-bit", lib.mx_gated, h["X"], *[lib.mx_empty(40, 300, "mx8", "cpu")] * 2, h["Y"])


def test_reference_quantisation():
    """Hand-made blocks: the largest entry decides the scale, ties go to even codes."""
    x = torch.zeros(1, 32)
    x[0, :8] = torch.tensor([6.99, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0])
    Q, S = ref.quantize(x, "mx4")
    assert S[0, 0] == 127 and [int(v) for v in ref.entries(Q, "mx4")[0, :8] * 2] == [12, 0, 2, 2, 4, 4, 8, -8]
    x[0, 0] = 7.0  # would round to 8: a larger scale
    Q, S = ref.quantize(x, "mx4")
    assert S[0, 0] == 128 and float(ref.values(Q, S, "mx4")[0, 0]) == 8.0
    x[0, :3] = torch.tensor([464.0, 2.0 ** -10, 3 * 2.0 ** -10])
    Q, S = ref.quantize(x, "mx8")
    assert S[0, 0] == 127 and [float(v) for v in ref.entries(Q, "mx8")[0, :3]] == [448.0, 0.0, 2.0 ** -8]
    x[0, 0] = float("inf")
    Q, S = ref.quantize(x, "mx8")
    assert S[0, 0] == 255 and not Q.any() and bool(torch.isnan(ref.values(Q, S, "mx8")[0, :32]).all())


def test_norm_gradients_against_differences():
    """The formula's gradients are those of finite differences of the norm's own 64-bit form."""
    g = torch.Generator().manual_seed(5)
    h, w, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((3, 40), (40,), (3, 40)))
    eps, d = 1e-6, 1e-6
    (dx, _), (dw, _) = ref.norm_backward(dy, h, w, None, eps)
    f = lambda a, b: float((ref.norm(a, None, b, eps)[1][0] * dy).sum())  # noqa: E731
    for i, j in ((0, 0), (1, 17), (2, 39)):
        for t, grad, at in ((h, dx, (i, j)), (w, dw, (j,))):
            p, q = t.clone(), t.clone()
            p[at] += d
            q[at] -= d
            slope = (f(p, w) - f(q, w) if t is h else f(h, p) - f(h, q)) / (2 * d)
            assert abs(slope - float(grad[at])) < 1e-7
