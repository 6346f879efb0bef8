"""The planner of the microscaled products (no GPU): the sizes that the GPU tests run reach every
compiled kernel, so that new estimates cannot leave one untested or without a call."""
import mx_shapes
from mx_planner import mx_planner  # noqa: F401
from software_pipelined_tiled_loop_amd import binding as lib

TYPES = (lib.PGEMM_F32, lib.PGEMM_F16, lib.PGEMM_BF16)


def test_the_tested_sizes_reach_every_kernel(mx_planner):  # noqa: F811
    queries = [(d, f, g) + s for s in mx_shapes.SHAPES for d in TYPES for f in (0, 1) for g in (0, 1)]
    variants, plans = mx_planner(queries)
    have = {(q[0], p[0]) for q, p in zip(queries, plans) if p[0] >= 0}
    assert set(variants) <= have, sorted(set(variants) - have)
    split = {(q[0], p[0]) for q, p in zip(queries, plans) if p[0] >= 0 and p[1] > 1}
    # splits of every size of tile, and of every format and pair among them
    assert {tuple(variants[i][k] for k in ("bm", "bn")) for i in split} >= {(256, 256), (256, 128), (128, 128), (128, 64),
                                                                            (16, 16), (16, 32), (32, 32), (64, 32)}
    assert {tuple(variants[i][k] for k in ("format", "gated")) for i in split} == {(0, 0), (0, 1), (1, 0), (1, 1)}
    for q, p in zip(queries, plans):
        assert p[0] < 0 or variants[q[0], p[0]]["format"] == q[1] and variants[q[0], p[0]]["gated"] == q[2]
        # many rows of MX8 with fp32 outputs go another way
        assert (p[0] < 0) == (q[0] == lib.PGEMM_F32 and q[1] == lib.MX8 and q[3] > 256), (q, p)


def test_launches_fit(mx_planner):  # noqa: F811
    """Every size that the checks let through has a launch, below 2^32 threads."""
    queries = [(lib.PGEMM_BF16, f, g, M, N, K) for f in (0, 1) for g in (0, 1) for K in (1, 256, 1 << 19)
               for M, N in ((1, (1 << 20) - 1), (1 << 20, 64), ((1 << 30) - 64, 1), (1 << 17, 1 << 18), (65536, 1 << 19))]
    _, plans = mx_planner(queries)
    for q, p in zip(queries, plans):
        assert p[0] >= 0 and 0 < p[2] < 1 << 32, (q, p)
