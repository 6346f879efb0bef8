"""What the assembly of the feed-forward kernels may not hold (no GPU), along every
path that a wave can take through a kernel (branches and loop back edges):

* a buffer store of 12 or 16 bytes whose scalar offset is a register: followed by a
  VALU write of its data, as the compiler places them, it stored wrong first dwords;
* a hazard around the MFMAs that are inline asm, which the compiler does not see: a
  VALU write of an A or B operand less than two wait states before the MFMA, or
  another access to an accumulator less than eighteen behind the MFMA that writes it;
* another write of M0 between the one that places an LDS-DMA load and the load.

Each scan is shown to find what is planted in a listing."""
import concurrent.futures as cf
import os
import re
import shutil
import subprocess

import pytest

from software_pipelined_tiled_loop_amd import build

UNITS = ("linear_bf16.hip", "linear_f16.hip", "linear_f32.hip")
OPERAND, ACCUMULATOR = 2, 18
REGISTER = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")


def parse(text):
    """(instructions, predecessors): each instruction's text, and where a wave may come from."""
    lines, labels = [], {}
    for raw in text.splitlines():
        line = raw.split(";")[0].strip()
        if re.match(r"^[.\w$]+:$", line):
            labels[line[:-1]] = len(lines)
        elif line and not line.startswith("."):
            lines.append(line)
    before = [[] for _ in lines]
    for i, line in enumerate(lines):
        op = line.split()[0]
        if op.startswith(("s_branch", "s_cbranch")):
            to = labels.get(line.split()[1])
            if to is not None and to < len(lines):
                before[to].append(i)
        assert not op.startswith(("s_setpc", "s_swappc", "s_call")), line
        if op not in ("s_branch", "s_endpgm") and i + 1 < len(lines):
            before[i + 1].append(i)
    return lines, before


def operands(line):
    parts = line.split(None, 1)
    return [p.strip() for p in parts[1].split(",")] if len(parts) > 1 else []


def registers(text):
    out = set()
    for kind, lo, hi, one in REGISTER.findall(text):
        out |= {(kind, int(one))} if one else {(kind, i) for i in range(int(lo), int(hi) + 1)}
    return out


def states(line):
    return int(line.split()[1], 0) + 1 if line.startswith("s_nop") else 1


def behind(lines, before, i, limit):
    """The instructions that can stand less than `limit` wait states before instruction i."""
    best, todo = {}, [(p, 0) for p in before[i]]
    while todo:
        p, gap = todo.pop()
        if gap >= limit or best.get(p, limit) <= gap:
            continue
        best[p] = gap
        todo += [(q, gap + states(lines[p])) for q in before[p]]
    return [lines[p] for p in best]


def wide_stores(lines, _):
    """Wide buffer stores with a scalar offset in a register."""
    found = []
    for line in lines:
        if re.match(r"buffer_store_(dwordx[34]|format_xyzw?|b96|b128)\b", line):
            at = operands(line)[3].split()[0]  # data, address, descriptor, scalar offset
            if not re.match(r"^(0x[0-9a-f]+|-?\d+)$", at):
                found.append(line)
    return found


def mfma_hazards(lines, before):
    found = []
    for i, line in enumerate(lines):
        mfma = line.startswith("v_mfma")
        if mfma and re.search(r" a\[", line):
            ops = operands(line)
            need, limit, writers = registers(ops[1]) | registers(ops[2]), OPERAND, False
        else:
            need = {r for r in registers(line) if r[0] == "a"}
            if mfma or not need:
                continue
            limit, writers = ACCUMULATOR, True
        for p in behind(lines, before, i, limit):
            if p.startswith("v_") and p.startswith("v_mfma") == writers and operands(p) and registers(operands(p)[0]) & need:
                found.append((p, line))
    return found


def lost_places(lines, before):
    """LDS-DMA loads that another write of M0 than the LDS address's can precede."""
    found = []
    for i, line in enumerate(lines):
        if not (line.startswith("buffer_load") and re.search(r"\blds$", line)):
            continue
        seen, todo = set(), list(before[i])
        if not todo:
            found.append(line)
        while todo:
            p = todo.pop()
            if p in seen:
                continue
            seen.add(p)
            ops = operands(lines[p])
            if ops and ops[0] == "m0":
                if not lines[p].startswith(("s_add_u32 m0,", "s_mov_b32 m0,")):
                    found.append((lines[p], line))
                continue
            if not before[p]:
                found.append(("no write of m0", line))
            todo += before[p]
    return found


def test_the_scans_find_what_is_planted():
    m = "v_mfma_f32_16x16x32_bf16 a[0:3], v[0:3], v[4:7], a[0:3]\n"
    assert wide_stores(*parse("buffer_store_dwordx4 v[0:3], v4, s[0:3], s9 offen"))
    assert wide_stores(*parse("buffer_store_dwordx3 v[0:2], v4, s[0:3], m0 offen offset:16"))
    assert not wide_stores(*parse("buffer_store_dwordx4 v[0:3], v4, s[0:3], 0 offen offset:16"))
    assert not wide_stores(*parse("buffer_store_dwordx2 v[0:1], v4, s[0:3], s9 offen"))
    assert mfma_hazards(*parse("v_mov_b32_e32 v5, v9\n" + m))
    assert not mfma_hazards(*parse("v_mov_b32_e32 v5, v9\ns_nop 1\n" + m))
    assert mfma_hazards(*parse(m + "s_nop 7\nv_accvgpr_read_b32 v0, a2"))
    assert not mfma_hazards(*parse(m + "s_nop 15\ns_nop 15\nv_accvgpr_read_b32 v0, a2"))
    # around a loop, and past a branch
    loop = ".L1:\n%s\ns_nop 15\ns_nop 15\n%s\ns_cbranch_scc1 .L1\ns_endpgm"
    assert mfma_hazards(*parse(loop % (m, "v_mov_b32_e32 v5, v9")))
    assert not mfma_hazards(*parse(loop % (m, "v_mov_b32_e32 v5, v9\ns_nop 1")))
    assert mfma_hazards(*parse(m + "s_branch .L2\ns_nop 15\ns_nop 15\n.L2:\nv_accvgpr_read_b32 v0, a2"))
    load = "buffer_load_dwordx4 v1, s[0:3], 0 offen lds"
    assert not lost_places(*parse("s_add_u32 m0, s1, 0x400\ns_nop 0\n" + load))
    assert lost_places(*parse("s_add_u32 m0, s1, 0x400\ns_movk_i32 m0, 7\n" + load))
    assert lost_places(*parse(load))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """(unit, name, parsed body) of every kernel that the library is built of."""
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
                found.append((unit, name, parse(rest[rest.index("\n"):rest.index("\n.Lfunc_end")])))
    assert len(found) >= 60 and {u for u, _, _ in found} == set(UNITS)
    return found


def test_no_wide_store_has_a_scalar_offset(kernels):
    stores = 0
    for unit, name, (lines, before) in kernels:
        stores += sum(line.startswith("buffer_store_dwordx4") for line in lines)
        assert not wide_stores(lines, before), (unit, name, wide_stores(lines, before)[:3])
    assert stores > 100


def test_no_hazard_around_the_asm_mfmas_on_any_path(kernels):
    asm = 0
    for unit, name, (lines, before) in kernels:
        # the tile kernels of 16-bit types; elsewhere the compiler knows its own MFMAs
        if "linear_kernel" in name and unit != "linear_f32.hip":
            asm += any(line.startswith("v_mfma") and " a[" in line for line in lines)
            found = mfma_hazards(lines, before)
            assert not found, (unit, name, found[:3])
    assert asm == 30  # three tile classes in five layouts, of both 16-bit types


def test_m0_reaches_its_load_on_every_path(kernels):
    loads = 0
    for unit, name, (lines, before) in kernels:
        loads += sum(line.startswith("buffer_load") and line.endswith("lds") for line in lines)
        found = lost_places(lines, before)
        assert not found, (unit, name, found[:3])
    assert loads > 1000
