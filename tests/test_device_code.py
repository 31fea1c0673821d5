"""Wait states that inline assembly owes, read from the disassembly of the built library.

The compiler does not look into an assembly string, so what it would put there itself has to be written there.  Between a
scalar write of M0 and a load into LDS, which takes its LDS address from M0, the architecture asks for one wait state; between
a vector instruction's write of a scalar register and a vector memory instruction that reads it, for five.
"""

import os
import re
import shutil
import subprocess

import pytest

from curvature_conditioned_query_amd.binding import library_path

OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
INSTRUCTION = re.compile(r"^\t([a-z]\w+)(?: (.*?))?\s*(?://.*)?$")
SCALARS = re.compile(r"\bs(?:(\d+)|\[(\d+):(\d+)\])")


def _scalars(text):
    """Numbers of the scalar registers that an operand names."""
    return {i for one, lo, hi in SCALARS.findall(text) for i in (range(int(one), int(one) + 1) if one else range(int(lo), int(hi) + 1))}


def missing_waits(lines):
    """(loads into LDS, those of them with too few wait states before them)."""
    m0, written = 9, {}  # wait states since M0 was written, and since each scalar register was by a vector instruction
    loads, short = 0, []
    for line in lines:
        m = INSTRUCTION.match(line)
        if m is None:
            continue
        name, operands = m.group(1), m.group(2) or ""
        if "_load_lds_" in name or (name.startswith("buffer_load") and operands.endswith(" lds")):
            loads += 1
            if m0 < 1 or any(written.get(s, 9) < 5 for s in _scalars(operands)):
                short.append(line.strip())
        passed = int(operands, 0) + 1 if name == "s_nop" else 1
        m0 += passed
        written = {s: n + passed for s, n in written.items() if n + passed < 5}
        first = operands.split(",")[0]
        if name.startswith("s_") and first == "m0":
            m0 = 0
        if name.startswith("v_"):
            # a scalar destination stands first (v_readfirstlane, v_cmp) or second (a carry out)
            targets = [first] if first.startswith("s") else operands.split(",")[1:2] if re.match(r"v_(add|sub|subrev)(c|b)?_co_|v_div_scale", name) else []
            for s in _scalars(" ".join(targets)):
                written[s] = 0
    return loads, short


def test_what_counts_as_a_missing_wait():
    load = "\tglobal_load_lds_dwordx4 v[0:1], off   // 0: 1"
    based = "\tglobal_load_lds_dwordx4 v0, s[4:5]"
    assert missing_waits(["\ts_mov_b32 m0, s3", load]) == (1, [load.strip()])
    assert missing_waits(["\ts_mov_b32 m0, s3", "\ts_nop 0", load]) == (1, [])
    assert missing_waits(["\ts_mov_b32 m0, s3", "\tv_add_u32_e32 v0, v1, v2", load, load]) == (2, [])
    assert missing_waits(["\tv_readfirstlane_b32 s5, v3", "\ts_mov_b32 m0, s3", "\ts_nop 0", based]) == (1, [based.strip()])
    assert missing_waits(["\tv_readfirstlane_b32 s5, v3", "\ts_mov_b32 m0, s3", "\ts_nop 3", based]) == (1, [])
    assert missing_waits(["\tv_readfirstlane_b32 s6, v3", "\ts_mov_b32 m0, s3", "\ts_nop 0", based]) == (1, [])


def test_loads_into_lds_wait_for_m0(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    path = tmp_path / "libccq.so"
    shutil.copy(library_path(), path)
    subprocess.run([OBJDUMP, "--offloading", str(path)], check=True, capture_output=True, cwd=tmp_path)
    parts = sorted(p for p in os.listdir(tmp_path) if p.endswith("gfx950"))
    assert parts
    loads, short = 0, []
    for p in parts:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", p], check=True, capture_output=True, text=True, cwd=tmp_path).stdout
        n, found = missing_waits(text.split("\n"))
        loads += n
        short += found
    assert loads > 100  # the prefill kernels and the walk of the linear attention
    assert not short, f"{len(short)} of {loads}: {short[:3]}"
