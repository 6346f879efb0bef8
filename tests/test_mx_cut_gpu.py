"""Products in 4 bits whose rows end with a group of scales of a single period, on the GPU: XCDs that begin in the middle of
the rows read the first group's scales right behind that period, and those of the groups differ by powers of two here."""
import pytest
import torch

import mx_reference as ref
from mx_cut_shapes import CUT
from software_pipelined_tiled_loop_amd import binding as pg

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def stored(g, rows, K, scale=1.0):
    """Random blocks, each group of 1024 entries of a size of its own, and their values."""
    x = torch.randn(rows, K, generator=g, device="cuda").mul_(scale)
    x *= torch.ldexp(torch.ones((), device="cuda"), torch.randint(-6, 1, (rows, -(-K // 1024)), generator=g, device="cuda")
                     ).repeat_interleave(1024, 1)[:, :K]
    mx = pg.mx_quantize(x, pg.mx_empty(rows, K, "mx4", "cuda"))
    return mx, pg.mx_dequantize(mx, torch.empty(rows, ref.filled(K), device="cuda")).double()


def check(got, v, e, t, what):
    v, e = ref.round_out(v, e, t)
    bad = ~((got.double() - v).abs() <= e)
    assert not bool(bad.any()), "%s %s: %d off, the first at %s" % (what, t, int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("M,N,K", CUT)
def test_rows_that_end_with_a_single_period(M, N, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N + K)
    X, x = stored(g, M, K)
    Wg, wg = stored(g, N, K, K ** -0.5)
    Wu, wu = stored(g, N, K, K ** -0.5)
    away = torch.empty(1 << 28, device="cuda")  # 1 GiB: puts the operands out of the caches
    for t in TYPES.values():
        (zg, eg), (zu, eu) = ref.product(x, wg, "mx4", t), ref.product(x, wu, "mx4", t)
        v, ev = ref.act_bound(zg, eg, "silu")
        h = v * zu
        for turn in range(3):
            away.fill_(turn)
            Y = pg.mx_linear(X, Wg, torch.full((M, N), 9.0, dtype=t, device="cuda"))
            check(Y, zg, eg, t, "linear")
            away.fill_(turn)
            H = pg.mx_gated(X, Wg, Wu, torch.full((M, N), 9.0, dtype=t, device="cuda"))
            check(H, h, ev * zu.abs() + v.abs() * eu + ev * eu + ref.S * h.abs(), t, "gated")
