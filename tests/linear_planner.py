"""The fixture `planner`: the planner of the feed-forward operators, asked on the host."""
import os
import shutil
import subprocess

import pytest

from software_pipelined_tiled_loop_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    """Runs linear_plans.cpp: (variants, choices of the queries given)."""
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    at = tmp_path_factory.mktemp("plans")
    # the planner and the table of variants are host code; the kernels' objects are the library's own
    sources = [os.path.join(build.CSRC, f) for f in os.listdir(build.CSRC) if f.endswith(".hpp") or f.startswith("linear_")]
    newest = max(os.path.getmtime(f) for f in sources)
    objs = []
    for name in ("linear_f32.hip", "linear_f16.hip", "linear_bf16.hip"):
        obj = os.path.join(build.BUILD_DIR, name + ".o")
        fresh = os.path.exists(obj) and os.path.getmtime(obj) >= newest
        objs.append(obj if fresh else build._compile(os.path.join(build.CSRC, name)))
    obj, exe = str(at / "plans.o"), str(at / "plans")
    flags = [f for f in build.HIPCC_FLAGS if f != "-O3"] + ["-O1"]
    for cmd in ([hipcc] + flags + ["-x", "hip", "-c", os.path.join(ROOT, "tests", "linear_plans.cpp"), "-o", obj],
                [hipcc, "--offload-arch=" + build.ARCH, obj] + objs + ["-o", exe]):
        subprocess.run(cmd, check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)

    def ask(queries):
        text = "".join("%d %d %d %d %d\n" % q for q in queries)
        out = subprocess.run([exe], input=text, stdout=subprocess.PIPE, text=True, check=True, timeout=300).stdout
        variants, plans = {}, []
        for line in out.splitlines():
            word, *n = line.split()
            n = tuple(map(int, n))
            if word == "variant":
                variants[n[:2]] = dict(zip(("lay", "gated", "few", "bm", "bn", "per_cu"), n[2:]))
            else:
                plans.append(n)
        assert len(plans) == len(queries)
        return variants, plans
    return ask
