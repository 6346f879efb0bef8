"""What the assembly of the microscaled products' kernels may not hold (no GPU), along every path that a
wave can take: wide buffer stores with a scalar offset in a register, hazards around the scaled MFMAs that are
inline asm (their scales are operands too), and another write of M0 between an LDS-DMA load's place and the load."""
import concurrent.futures as cf
import os
import re
import shutil
import subprocess

import pytest

from software_pipelined_tiled_loop_amd import build
from test_linear_assembly import behind, lost_places, operands, parse, registers, wide_stores

UNITS = ("mx_bf16.hip", "mx_f16.hip", "mx_f32.hip")
OPERAND, ACCUMULATOR = 2, 20  # wait states; the scaled MFMAs take at most sixteen passes


def scaled_hazards(lines, before):
    found = []
    for i, line in enumerate(lines):
        mfma = line.startswith("v_mfma")
        if mfma and re.search(r" a\[", line):
            ops = operands(line)
            scales = registers(ops[4]) | registers(ops[5].split()[0]) if line.startswith("v_mfma_scale") else set()
            need, limit, writers = registers(ops[1]) | registers(ops[2]) | scales, OPERAND, False
        else:
            need = {r for r in registers(line) if r[0] == "a"}
            if mfma or not need:
                continue
            limit, writers = ACCUMULATOR, True
        for p in behind(lines, before, i, limit):
            if p.startswith("v_") and p.startswith("v_mfma") == writers and operands(p) and registers(operands(p)[0]) & need:
                found.append((p, line))
    return found


def test_the_scan_finds_what_is_planted():
    m = ("v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], v[0:3], v[4:7], a[0:3], v20, v21 op_sel:[0,0,0] op_sel_hi:[0,0,0] "
         "cbsz:4 blgp:4\n")
    for at in (5, 20, 21):
        assert scaled_hazards(*parse("v_mov_b32_e32 v%d, v9\n" % at + m))
        assert not scaled_hazards(*parse("v_mov_b32_e32 v%d, v9\ns_nop 1\n" % at + m))
    assert not scaled_hazards(*parse("v_mov_b32_e32 v22, v9\n" + m))
    assert scaled_hazards(*parse(m + "s_nop 15\nv_accvgpr_read_b32 v0, a2"))
    assert not scaled_hazards(*parse(m + "s_nop 15\ns_nop 15\nv_accvgpr_read_b32 v0, a2"))
    assert scaled_hazards(*parse(".L1:\n%s\ns_nop 15\ns_nop 15\nv_mov_b32_e32 v20, v9\ns_cbranch_scc1 .L1\ns_endpgm" % m))
    assert scaled_hazards(*parse(".L1:\n%s\ns_nop 15\ns_nop 15\ns_cbranch_scc0 .L2\nv_mov_b32_e32 v20, v9\n.L2:\n%s" % (m, m)))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """(unit, name, parsed body, metadata) of every kernel of the norm and the microscaled operators."""
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    at = tmp_path_factory.mktemp("assembly")

    def compile_unit(unit):
        out = str(at / (unit + ".s"))
        subprocess.run([hipcc] + build.HIPCC_FLAGS + ["--cuda-device-only", "-S", os.path.join(build.CSRC, unit), "-o", out],
                       check=True, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        with open(out) as f:
            return f.read()

    with cf.ThreadPoolExecutor(max_workers=len(UNITS)) as ex:
        texts = list(ex.map(compile_unit, UNITS))
    found = []
    for unit, text in zip(UNITS, texts):
        for body in re.split(r"\n(?=_ZN5pgemm\S+:)", text)[1:]:
            name, rest = body.split(":", 1)
            if ".Lfunc_end" in rest:
                found.append((unit, name, parse(rest[rest.index("\n"):rest.index("\n.Lfunc_end")]),
                              int(re.search(r"\.amdhsa_private_segment_fixed_size (\d+)", rest).group(1))))
    assert len(found) >= 100 and {u for u, _, _, _ in found} == set(UNITS)
    return found


def test_no_wide_store_has_a_scalar_offset(kernels):
    for unit, name, (lines, before), _ in kernels:
        assert not wide_stores(lines, before), (unit, name, wide_stores(lines, before)[:3])


def test_no_hazard_around_the_asm_mfmas_on_any_path(kernels):
    asm = 0
    for unit, name, (lines, before), _ in kernels:
        if "mx_tile" in name or "mx_large" in name:  # elsewhere the compiler knows its own MFMAs
            asm += any(line.startswith("v_mfma_scale") and " a[" in line for line in lines)
            found = scaled_hazards(lines, before)
            assert not found, (unit, name, found[:3])
    assert asm == 20  # two tile classes, gated or not, of both formats (fp32 outputs: of MX4)


def test_m0_reaches_its_load_on_every_path(kernels):
    loads = 0
    for unit, name, (lines, before), _ in kernels:
        loads += sum(line.startswith("buffer_load") and line.endswith("lds") for line in lines)
        found = lost_places(lines, before)
        assert not found, (unit, name, found[:3])
    assert loads > 500


def test_nothing_spills(kernels):
    for unit, name, _, scratch in kernels:
        assert scratch == 0, (unit, name, scratch)
