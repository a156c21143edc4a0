"""The machine code of the built library (CPU only): a load that goes straight to LDS takes its
LDS address from M0, and the hardware asks for one wait state between a scalar write of M0 and
such a load.  The compiler keeps to that for its own instructions, not inside hand-written ones.
"""
import os
import re
import shutil
import subprocess

import pytest

from test_operator_refusals import L  # noqa: F401

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
TO_LDS = re.compile(r"^(global|scratch)_load_lds_|^buffer_(load|store)_.*\blds\b")


def instructions(lib, folder):
    """Each kernel's instructions in order, as text, over all code objects of the library."""
    copy = shutil.copy(lib, folder)
    subprocess.run([OBJDUMP, "--offloading", copy], cwd=folder, check=True, capture_output=True)
    objects = sorted(f for f in os.listdir(folder) if "amdgcn" in f)
    assert objects
    for f in objects:
        out = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", f], cwd=folder, check=True, capture_output=True, text=True).stdout
        for line in out.splitlines():
            yield line.split("//")[0].strip()


def short_of_wait(lines):
    """(loads to LDS, those that follow a write of M0 at once)."""
    loads, short, before = 0, [], ""
    for line in lines:
        if TO_LDS.match(line):
            loads += 1
            if before.startswith("s_") and re.match(r"s_\w+ m0\b", before):
                short.append((before, line))
        if line:
            before = line
    return loads, short


def test_the_search_finds_what_it_looks_for():
    load = "global_load_lds_dwordx4 v1, s[2:3]"
    assert short_of_wait(["s_mov_b32 m0, s4", load]) == (1, [("s_mov_b32 m0, s4", load)])
    assert len(short_of_wait(["s_add_i32 m0, s4, 0x400", "", "buffer_load_dword v1, s[4:7], 0 offen lds"])[1]) == 1
    assert short_of_wait(["s_mov_b32 m0, s4", "s_nop 0", load, "s_mov_b32 s5, m0", load]) == (2, [])


def test_no_load_to_lds_right_behind_a_write_of_m0(L, tmp_path):  # noqa: F811
    if not os.path.exists(OBJDUMP):
        pytest.skip("needs the compiler's llvm-objdump")
    loads, short = short_of_wait(instructions(L.LIB_PATH, tmp_path))
    assert loads > 100 and not short, (loads, len(short), short[:3])
