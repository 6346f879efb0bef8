"""What the K loops of the microscaled products read has arrived (no GPU): mx_loads.cpp walks along the kernels' loads,
edges and reads for every stored length up to 40960 entries, every place in a row that an XCD begins at, and every split.
And the sizes that the GPU tests run for rows whose last group of scales is a single period do take those kernels."""
import os
import re
import shutil
import subprocess

import pytest

from mx_cut_shapes import CUT, FEW, FEW_SPLIT, LARGE, LARGE_SPLIT, TILE, TILE_SPLIT
from mx_planner import mx_planner  # noqa: F401
from software_pipelined_tiled_loop_amd import binding as lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    exe = str(tmp_path_factory.mktemp("mx_loads") / "walk")
    subprocess.run([hipcc, "-O2", "-std=c++17", "-Wno-inline-asm", "--offload-arch=gfx950", "--cuda-host-only", "-x", "hip",
                    "-I" + os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "mx_loads.cpp"), "-o", exe],
                   check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    return lambda *a: subprocess.run([exe, *a], stdout=subprocess.PIPE, text=True, timeout=300).stdout.strip()


def test_every_read_is_covered(walk):
    out = walk()
    assert re.match(r"^OK \d{8,}$", out), out


def test_the_walk_finds_a_wait_that_is_too_short(walk):
    """Edge Y that leaves the scales under way: rows of 1024 n + 256 stored entries, from three groups on."""
    assert [int(e) for e in walk("mistaken").split()] == list(range(2304, 40961, 1024))


def test_cut_groups_take_the_large_tiles(mx_planner):  # noqa: F811
    """In 4 bits, whole, of both products and of every type of output."""
    queries = [(d, lib.MX4, g) + s for s in CUT for d in (lib.PGEMM_F32, lib.PGEMM_F16, lib.PGEMM_BF16) for g in (0, 1)]
    variants, plans = mx_planner(queries)
    for q, (index, splits, _) in zip(queries, plans):
        v = variants[q[0], index]
        assert v["bm"] == 256 and splits == 1 and -(-q[5] // 256) % 4 == 1 and q[5] > 2048, (q, v, splits)


def test_places_take_a_kernel_of_each_kind(mx_planner):  # noqa: F811
    """The sizes at which rows of blocks lie apart, and at which calls are repeated."""
    for shape, rows, whole in ((FEW, range(16, 65), True), (FEW_SPLIT, range(16, 65), False), (TILE, (128,), True),
                               (TILE_SPLIT, (128, 256), False), (LARGE, (256,), True), (LARGE_SPLIT, (256,), False)):
        queries = [(d, f, g) + shape for d in (lib.PGEMM_F16, lib.PGEMM_BF16) for f in (0, 1) for g in (0, 1)]
        variants, plans = mx_planner(queries)
        for q, (index, splits, _) in zip(queries, plans):
            assert variants[q[0], index]["bm"] in rows and (splits == 1) == whole, (q, variants[q[0], index], splits)
            assert shape != TILE_SPLIT or q[2] or variants[q[0], index]["bm"] == 128
