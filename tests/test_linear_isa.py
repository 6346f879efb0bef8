"""The lone-wave tile's MFMAs are inline asm, so the compiler keeps none of their
hazards away.  This scans the assembly of the library's own kernels for them
(no GPU): a VALU write of an MFMA's A or B operand less than two wait states
before it, and any other access to an accumulator less than eighteen behind the
MFMA that writes it."""
import os
import re
import shutil
import subprocess

import pytest

from software_pipelined_tiled_loop_amd import build

OPERAND, ACCUMULATOR = 2, 18


def registers(text):
    out = set()
    for kind, lo, hi, kind1, one in re.findall(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        if kind:
            out |= {(kind, i) for i in range(int(lo), int(hi) + 1)}
        else:
            out.add((kind1, int(one)))
    return out


def operands(line):
    parts = line.split(None, 1)
    return [p for p in parts[1].split(",")] if len(parts) > 1 else []


def states(line):
    return int(line.split()[1]) + 1 if line.startswith("s_nop") else 1


def scan(lines):
    """Hazards of one kernel, and its MFMAs with AGPR accumulators."""
    found, count = [], 0
    for i, line in enumerate(lines):
        mfma = line.startswith("v_mfma")
        if mfma and " a[" in line:
            count += 1
            ops = operands(line)
            need, limit = registers(ops[1]) | registers(ops[2]), OPERAND
        else:
            need, limit = {r for o in operands(line) for r in registers(o) if r[0] == "a"}, ACCUMULATOR
            if mfma or not need:
                continue
        gap = 0
        for p in reversed(lines[max(0, i - 40):i]):
            if gap >= limit:
                break
            writes = registers(operands(p)[0]) if p.startswith("v_") and operands(p) else set()
            if p.startswith("v_mfma") != (limit == OPERAND) and writes & need:
                found.append((p, line))
                break
            gap += states(p)
    return found, count


def test_scan_sees_planted_hazards():
    m = "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]"
    assert scan(["v_mov_b32_e32 v5, v9", m])[0]
    assert not scan(["v_mov_b32_e32 v5, v9", "s_nop 1", m])[0]
    assert scan([m, "s_nop 7", "v_accvgpr_read_b32 v0, a2"])[0]
    assert not scan([m, "s_nop 15", "s_nop 15", "v_accvgpr_read_b32 v0, a2"])[0]


@pytest.mark.parametrize("unit", ["linear_bf16.hip", "linear_f16.hip"])
def test_no_hazard_around_the_lone_mfmas(unit, tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    with open(os.path.join(build.CSRC, unit)) as f:
        tiles = re.findall(r"LIN_CLASS\(DT_\w+, [^)]*\)", f.read())
    src, out = tmp_path / "tile.hip", str(tmp_path / "tile.s")
    src.write_text('#include "linear_variants.hpp"\nnamespace pgemm { LinVariant tile[] = {%s}; }\n' % ", ".join(tiles))
    subprocess.run([hipcc] + build.HIPCC_FLAGS + ["-I" + build.CSRC, "--cuda-device-only", "-S", str(src), "-o", out],
                   check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    with open(out) as f:
        text = f.read()
    kernels = 0
    for body in re.split(r"\n(?=_ZN5pgemm13linear_kernel\S+:)", text)[1:]:
        name = body.split(":", 1)[0]
        lines = [ln.split(";")[0].strip() for ln in body[:body.find(".Lfunc_end")].splitlines() if ln.startswith("\t")]
        found, count = scan([ln for ln in lines if ln and not ln.startswith(".")])
        assert not found, (name, found[:3])
        kernels += count > 0
    assert kernels == 5 * len(tiles)  # each tile in every layout
