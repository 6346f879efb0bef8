"""No launch of the feed-forward operators has more threads than a grid holds (2^32):
the planner takes another kernel, or the call is refused (no GPU)."""
import random

from linear_planner import planner  # noqa: F401
from software_pipelined_tiled_loop_amd import binding as lib

TYPES = (lib.PGEMM_F32, lib.PGEMM_F16, lib.PGEMM_BF16)
LARGE = -7


def test_every_choice_fits_a_launch(planner):
    rng = random.Random(1)
    queries = [(d, k, M, N, K) for d in TYPES for k in range(12) for M, N, K in (
        (837248577, 132, 10), (653395173, 161, 4), (546360210, 135, 3), (1 << 29, 64, 8), (1 << 29, 1, 1), (1 << 30, 1, 1),
        (5, 1 << 20, 1 << 15))]
    queries += [(rng.choice(TYPES), rng.randrange(12), int(2 ** rng.uniform(0, 30))) + tuple(
        int(2 ** rng.uniform(0, 21)) for _ in range(2))
                for _ in range(3000)]
    queries = [q for q in queries if lib.pgemm_linear_workspace(*q[2:], q[0]) >= 0]
    assert len(queries) > 1500
    _, plans = planner(queries)
    for q, p in zip(queries, plans):
        assert p[0] < 0 or p[2] < 1 << 32, (q, p)


def test_sizes_beyond_a_launch_are_refused():
    """The pass over dZ's 64 x 128 pieces would have 2^32 threads and more."""
    for M, N, K in ((546360210, 135, 3), (653395173, 161, 4)):
        for d in TYPES:
            assert lib.pgemm_gated_backward_workspace(M, N, K, d) == LARGE
            assert lib.pgemm_linear_backward_workspace(M, N, K, 2, d) == LARGE
            fake = 1 << 20
            assert lib.pgemm_linear_backward(M, N, K, fake, N, fake, K, fake, N, 0, fake, N, 2, fake, K, None, N, 0, None, d, d,
                                             fake, 1 << 50, None) == LARGE
    for M, N, K in ((1 << 29, 64, 8), (1 << 28, 128, 128), (100, 1 << 20, 1 << 15)):
        assert lib.pgemm_linear_backward_workspace(M, N, K, 2, 0) > 0
        assert lib.pgemm_gated_workspace(M, N, K, 2) >= 0
