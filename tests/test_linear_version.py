"""The ABI's version counts the feed-forward operators (no GPU)."""
import os
import re

from software_pipelined_tiled_loop_amd import binding as lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_version_and_exports():
    assert lib.pgemm_version() == 10100  # major * 10000 + minor * 100 + patch
    with open(os.path.join(ROOT, "include", "pgemm.h")) as f:
        names = set(re.findall(r"^\w+ (pgemm_(?:linear|gated)\w*)\(", f.read(), re.M))
    assert names == {p + q + r for p in ("pgemm_linear", "pgemm_gated") for q in ("", "_backward") for r in ("", "_workspace")}
    for name in names:
        assert hasattr(lib._lib, name)
