"""The instances of the per-head norms in the compiled code: those that the dispatch reaches."""

import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from rotation_activation_quantization_amd import build as B

SOURCES = ("qk_norm_rope.hip",)


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


def test_no_instance_of_the_norms_that_no_call_reaches(code):
    """Partners in another lane (1) need two lanes a head, those in whole chunks elsewhere in it (2) four."""
    names = [k for k in code["qk_norm_rope.hip"] if "qk_norm_rope_kernel" in k]
    assert len(names) == 78
    for name in names:
        lanes, pairs = (int(v) for v in re.search(r"kernelILi(\d+)ELb\dELb\dELi(\d)E", name).groups())
        assert lanes > {1: 1, 2: 2}.get(pairs, 0), name
