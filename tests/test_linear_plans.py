"""The planner of the feed-forward operators (no GPU): the sizes that the GPU tests run
reach every compiled kernel, so that new estimates cannot leave one untested."""
import linear_shapes
from linear_planner import planner  # noqa: F401
from software_pipelined_tiled_loop_amd import binding as lib

TYPES = (lib.PGEMM_F32, lib.PGEMM_F16, lib.PGEMM_BF16)


def group(kind):
    """Products that differ in more than a kernel's arguments: dW's stored order does not."""
    return kind if kind < 8 else 8 + (kind - 8) // 2 * 2


def test_the_tested_sizes_reach_every_tile_class_whole_and_split(planner):
    queries = [(d,) + s for s in linear_shapes.TILES for d in TYPES]
    variants, plans = planner(queries)
    have = {(q[0], group(q[1]), p[0], p[1] > 1) for q, p in zip(queries, plans)}
    need = set()
    for (d, i), v in variants.items():
        if v["few"]:
            continue
        kinds = {(0, 0): (0, 5, 7), (1, 0): (1, 4, 6), (2, 0): (8, 10), (0, 1): (2,), (1, 1): (3,)}[v["lay"], v["gated"]]
        need |= {(d, k, i, split) for k in kinds for split in (False, True)}
    assert len(need) == 160 and need <= have, sorted(need - have)
    assert all(n % 8 for s in linear_shapes.TILES for n in s[1:] if n > 8)


def test_the_tested_sizes_reach_every_few_rows_kernel(planner):
    queries = [(d,) + s for s in linear_shapes.FEW for d in TYPES]
    variants, plans = planner(queries)
    have = {(q[0], p[0], p[1] > 1) for q, p in zip(queries, plans)}
    need = {(d, i, split) for (d, i), v in variants.items() if v["few"] for split in (False, True)}
    assert need <= have, sorted(need - have)
