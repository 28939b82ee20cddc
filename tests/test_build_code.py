"""What the compiled products have to keep in order beyond what the compiler knows: the readers of a sum that matrix
instructions in inline assembly form, and loads to a place of LDS that reads have just left.  Checked on the assembly
along every path.  And the instances of the per-head norms: those that the dispatch reaches."""

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from rotation_activation_quantization_amd import build as B

SOURCES = ("linear_mx.hip", "linear_w8.hip", "qk_norm_rope.hip")
# wait states from a matrix instruction of sixteen passes to a reader of its result, and one to spare
SETTLED = 20


def assembly(src):
    cmd = [B.hipcc(), *B.COMMON, "-x", "hip", "--cuda-device-only", "-S", os.path.join(B.CSRC, src), "-o", "-"]
    return subprocess.run(cmd, capture_output=True, text=True, check=True).stdout


def functions(text):
    """{mangled name: lines of instructions and labels}"""
    out, lines = {}, None
    for line in text.splitlines():
        start = re.match(r"(_Z\w+):", line)
        if start:
            lines = out.setdefault(start[1], [])
        elif line.startswith(".Lfunc_end"):
            lines = None
        elif lines is not None:
            line = line.split(";")[0].strip()
            if line.startswith(".LBB") or (line and line[0] not in ".;#"):
                lines.append(line)
    return out


@pytest.fixture(scope="module")
def code():
    with ThreadPoolExecutor(len(SOURCES)) as pool:
        return {s: functions(t) for s, t in zip(SOURCES, pool.map(assembly, SOURCES))}


def blocks_of(lines):
    """(blocks of instructions, successors of each)"""
    blocks, at, cur = [[]], {}, 0
    for line in lines:
        if line.endswith(":"):
            if blocks[cur]:
                blocks.append([])
                cur += 1
            at[line[:-1]] = cur
            continue
        blocks[cur].append(line)
        if line.startswith(("s_branch", "s_cbranch", "s_endpgm")):
            blocks.append([])
            cur += 1
    after = []
    for n, b in enumerate(blocks):
        last = b[-1] if b else ""
        to = [at[last.split()[-1]]] if last.startswith(("s_branch", "s_cbranch")) else []
        if not last.startswith(("s_branch", "s_endpgm")) and n + 1 < len(blocks):
            to.append(n + 1)
        after.append(to)
    return blocks, after


def flow(lines, start, step, join):
    """Runs step(state, instruction) -> state over every path, from join over what comes into a block."""
    blocks, after = blocks_of(lines)
    into, todo = {0: start}, [0]
    while todo:
        n = todo.pop()
        state = into[n]
        for line in blocks[n]:
            state = step(state, line)
        for m in after[n]:
            new = state if m not in into else join(into[m], state)
            if m not in into or new != into[m]:
                into[m] = new
                todo.append(m)


def registers(text):
    out = set()
    for a, b, one in re.findall(r"\bv(?:\[(\d+):(\d+)\]|(\d+))", text):
        out.update(range(int(a), int(b) + 1) if a else (int(one),))
    return out


def unsettled(lines):
    """Instructions that touch a sum before the matrix instruction that forms it has ended."""
    bad = []

    def step(ages, line):
        name, _, rest = line.partition(" ")
        states = int(rest, 0) + 1 if name == "s_nop" else 1
        operands = rest.split(",")
        if name.startswith("v_mfma"):
            dest, source = registers(operands[0]), registers(rest)
            assert registers(",".join(re.findall(r"v\[\d+:\d+\]|v\d+", rest)[3:4])) == dest, line  # sums in place
            read = source - dest
        else:
            dest, read = set(), registers(rest)
        bad.extend([line] * bool(read & ages.keys()))
        ages = {r: a + states for r, a in ages.items() if a + states < SETTLED}
        ages.update(dict.fromkeys(dest, 0))
        return ages

    def join(a, b):
        return {r: min(a.get(r, SETTLED), b.get(r, SETTLED)) for r in a.keys() | b.keys()}

    flow(lines, {}, step, join)
    return bad


def early_loads(lines):
    """Loads to LDS issued while reads of LDS may still be on their way."""
    bad = []

    def step(reading, line):
        if line.startswith("ds_read"):
            return True
        if line.startswith("s_waitcnt"):
            return reading and "lgkmcnt(0)" not in line
        if reading and re.search(r"_load\w*_lds|_load.*\blds$", line):
            bad.append(line)
        return reading

    flow(lines, False, step, lambda a, b: a or b)
    return bad


def test_the_checks_see_what_they_look_for():
    mfma = "v_mfma_scale_f32_16x16x128_f8f6f4 v[4:7], v[8:11], v[12:15], v[4:7], v1, v2 cbsz:4 blgp:4"
    assert unsettled([mfma, "s_nop 15", "v_add_f32_e32 v0, v0, v5"])
    assert not unsettled([mfma, "s_nop 15", "s_nop 15", "v_add_f32_e32 v0, v0, v5"])
    assert unsettled([mfma, "v_mov_b32_e32 v6, 0"])
    assert unsettled([".LBB0_1:", "ds_write_b128 v0, v[4:7]", mfma, "s_cbranch_scc1 .LBB0_1", "s_endpgm"])
    load = "buffer_load_dwordx4 v60, s[0:3], s16 offen lds"
    assert early_loads(["ds_read_b128 v[0:3], v4", load])
    assert early_loads([".LBB0_1:", load, "ds_read_b128 v[0:3], v4", "s_cbranch_scc1 .LBB0_1", "s_endpgm"])
    assert early_loads(["ds_read_b128 v[0:3], v4", "s_waitcnt lgkmcnt(1)", "global_load_lds_dword v[60:61], off"])
    assert not early_loads(["ds_read_b128 v[0:3], v4", "s_waitcnt vmcnt(0) lgkmcnt(0)", load])


def test_sums_are_read_when_they_are_there(code):
    kernels = {k: v for k, v in code["linear_mx.hip"].items() if "mx_tile_kernel" in k}
    assert len(kernels) == 10
    for name, lines in kernels.items():
        assert any(line.startswith("v_mfma_scale") for line in lines)
        assert not unsettled(lines), name


@pytest.mark.parametrize("src,kernel", [("linear_mx.hip", "mx_few_kernel"), ("linear_w8.hip", "w8_few_kernel")])
def test_a_slot_is_loaded_when_its_reads_are_done(code, src, kernel):
    kernels = {k: v for k, v in code[src].items() if kernel in k}
    assert len(kernels) == 8
    for name, lines in kernels.items():
        assert sum(bool(re.search(r"\blds$|_load_lds", line)) for line in lines) and sum("ds_read" in x for x in lines)
        assert not early_loads(lines), name


def test_no_instance_of_the_norms_that_no_call_reaches(code):
    """Partners in another lane (1) need two lanes a head, those in whole chunks elsewhere in it (2) four."""
    names = [k for k in code["qk_norm_rope.hip"] if "qk_norm_rope_kernel" in k]
    assert len(names) == 78
    for name in names:
        lanes, pairs = (int(v) for v in re.search(r"kernelILi(\d+)ELb\dELb\dELi(\d)E", name).groups())
        assert lanes > {1: 1, 2: 2}.get(pairs, 0), name
