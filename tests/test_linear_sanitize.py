"""Address and undefined-behaviour sanitizers on the host code of the feed-forward
operators (no GPU): linear_sanitize.cpp drives the choice of tiles and splits and
the argument checks.  linear_abi.cpp and the driver are built with the sanitizers
on the host side only (each flag behind -Xarch_host); the kernels are the
library's own objects."""
import os

import pytest

from software_pipelined_tiled_loop_amd import build
from test_sanitizers import ENV, HOST_SAN, ROOT, _run


def test_linear_host_paths_under_sanitizers(tmp_path):
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    objs = []
    for name in ("linear_f32.hip", "linear_f16.hip", "linear_bf16.hip"):
        src = os.path.join(build.CSRC, name)
        built = os.path.join(build.BUILD_DIR, name + ".o")
        fresh = os.path.exists(built) and os.path.getmtime(built) >= os.path.getmtime(src)
        objs.append(built if fresh else build._compile(src))
    flags = [f for f in build.HIPCC_FLAGS if f != "-O3"] + ["-O1", "-g"]
    for src in (os.path.join(build.CSRC, "linear_abi.cpp"), os.path.join(ROOT, "tests", "linear_sanitize.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([hipcc] + flags + HOST_SAN + ["-x", "hip", "-c", src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "linear_sanitize")
    _run([hipcc, "--offload-arch=" + build.ARCH] + HOST_SAN + objs + ["-o", exe])
    out = _run([exe], env=ENV, timeout=600)
    assert out.strip().splitlines()[-1].startswith("OK"), out[-2000:]
