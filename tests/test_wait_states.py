"""Wait states that the instruction set asks of a program and that the compiler adds by itself, but
not inside an asm block: read from the machine code of the built library (no GPU needed).

A load straight into LDS takes its LDS address from m0. Between a scalar instruction that writes m0
and such a load one wait state has to pass, and five between a vector instruction that writes a
scalar register and a memory instruction that reads it (the load's buffer descriptor). With fewer
the load may see the register's old value: here, put 1 KB of a tile at another LDS address."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from selective_scan_amd import build, ops

OBJDUMP = os.path.join(os.path.dirname(build.HIPCC), "..", "llvm", "bin", "llvm-objdump")


def _scalars(operands):
    out = set()
    for one, lo, hi in re.findall(r"\bs(\d+)\b|\bs\[(\d+):(\d+)\]", operands):
        out |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def _states(ins):
    """Wait states that an instruction takes."""
    return int(ins.split()[1], 0) + 1 if ins.startswith("s_nop ") else 1


def violations(instructions):
    """(loads into LDS, [the too early ones]) of a list of instructions in program order."""
    loads, early = 0, []
    for i, ins in enumerate(instructions):
        if not re.match(r"(buffer|global|scratch)_load_.*\blds\b", ins):
            continue
        loads += 1
        reads, passed = _scalars(ins), 0
        for before in reversed(instructions[max(0, i - 5):i]):
            writes = before.split(None, 1)[1].split(",")[0] if " " in before else ""
            if passed < 1 and before.startswith("s_") and writes == "m0":
                early.append((before, ins))
            if passed < 5 and before.startswith("v_") and _scalars(writes) & reads:
                early.append((before, ins))
            passed += _states(before)
    return loads, early


@pytest.mark.parametrize("before,good", [
    (["s_mov_b32 m0, s2"], False),
    (["s_add_i32 m0, s2, 0x400"], False),
    (["s_mov_b32 m0, s2", "s_nop 0"], True),
    (["s_mov_b32 m0, s2", "v_add_u32_e32 v1, v2, v3"], True),
    (["v_readfirstlane_b32 s6, v3", "s_mov_b32 m0, s2", "s_nop 0"], False),
    (["v_readfirstlane_b32 s6, v3", "s_mov_b32 m0, s2", "s_nop 3"], True),
    (["v_readfirstlane_b32 s9, v3", "s_mov_b32 m0, s2", "s_nop 0"], True),
])
def test_the_check_itself(before, good):
    loads, early = violations(before + ["buffer_load_dwordx4 v3, s[4:7], 0 offen lds"])
    assert loads == 1 and (not early) == good


def test_loads_into_lds_wait_for_their_address(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump beside hipcc")
    ops.lib()
    copy = shutil.copy(build.LIB, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", copy], check=True, capture_output=True, cwd=tmp_path)
    loads = 0
    for obj in glob.glob(f"{copy}.*gfx950"):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", obj], check=True, capture_output=True,
                              text=True).stdout
        code = [t for t in (l.split("//")[0].strip() for l in text.splitlines()) if re.match(r"[a-z]\w+( |$)", t)]
        n, early = violations(code)
        loads += n
        assert not early, f"{len(early)} of {n} loads, the first: {early[0]}"
    assert loads > 0
