"""Smooth activations and their slopes far below zero, relative to the value.

The bias carries the values (a product over zeros adds nothing), fp32 outputs show
them unrounded.  Bounds, s = 2^-24: the exponential's argument a (silu |x|, gelu
x^2 / 2, gelu_tanh 2 sqrt(2/pi) (|x| + 0.044715 |x|^3)) is the result of at most four
roundings, so exp is off by 4 a s; exp2, the reciprocal and the fit (9e-8 < 2 s) by
2 s each, the polynomial and the products around them by at most 12 s more: the
value by (4 a + 20) s relative.  A slope is a sum Phi + x phi (silu, gelu_tanh: p + x p
(1 - p) (x P)') whose two terms carry that each.  Reciprocals below fp32's smallest
normal are zero: 128 * 2^-126 absolutely.
"""
import math

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
S = ref.S
FLUSH = 2.0 ** -119


@pytest.fixture(scope="module")
def pg():
    from software_pipelined_tiled_loop_amd import binding
    return binding


def argument(x, act):
    if act == "silu":
        return x.abs()
    if act == "gelu":
        return 0.5 * x * x
    return 2 * math.sqrt(2 / math.pi) * (x.abs() + 0.044715 * x.abs() ** 3)


def exact(x, act):
    """act(x), and the two terms of act'(x), without cancellation."""
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-x / math.sqrt(2))  # accurate far below zero too
        return x * p, p, x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == "silu":
        p, inner = torch.special.expit(x), torch.ones_like(x)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        p, inner = torch.special.expit(c * (x + 0.044715 * x ** 3)), c * (1 + 3 * 0.044715 * x * x)
    return x * p, p, x * p * (1 - p) * inner


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_values_and_slopes_relative_to_themselves(pg, dtype, act):
    print("[case] tails", dtype, act, flush=True)
    t, n = TYPES[dtype], 4096
    low = {"silu": -80.0, "gelu": -12.5, "gelu_tanh": -9.0}[act]
    z = torch.linspace(low, 6.0, n).to(t).cuda()
    x0, w0 = torch.zeros(1, 16, dtype=t, device="cuda"), torch.zeros(16, n, dtype=t, device="cuda")
    y = torch.empty(1, n, device="cuda")
    pg.linear(x0, w0, y, bias=z, act=act)
    one, db = torch.ones(1, n, dtype=t, device="cuda"), torch.empty(n, device="cuda")
    pg.linear_backward(one, x0, w0, Z=z.view(1, n), act=act, dbias=db)
    x = z.double().cpu()
    v, p, q = exact(x, act)
    rel = (4 * argument(x, act) + 20) * S
    ref.check("act", y[0], (v, rel * v.abs() + FLUSH))
    ref.check("slope", db, (p + q, rel * (p.abs() + q.abs()) + FLUSH))
