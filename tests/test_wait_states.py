"""Wait states around the direct HBM -> LDS loads (CPU: the built library is
disassembled, nothing runs).

These loads are issued from inline assembly, which the compiler's hazard pass
does not look into.  On gfx950 a load to LDS needs one wait state after a
scalar write of M0, and five between a vector instruction that writes a scalar
register and a vector memory instruction that takes its address from it.  An
instruction counts as one wait state, s_nop n as n + 1; a label ends the look
back (the code before it is not known to run).
"""

import os
import re
import shutil
import subprocess

import pytest

import expanded_dispatch_layout_amd as M

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump"))
                if p and os.path.exists(p)), None)


def _disassembly(tmp):
    lib = shutil.copy(M.LIB_PATH, tmp)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp, check=True, capture_output=True)
    for f in sorted(os.listdir(tmp)):
        if "gfx950" in f:
            yield from subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", f], cwd=tmp,
                                      check=True, capture_output=True,
                                      text=True).stdout.splitlines()


def hazards(lines):
    """(loads to LDS seen, the ones that come too early)."""
    seen, early, before = 0, [], []
    for line in lines:
        if re.match(r"^[0-9a-f]+ <.*>:$", line):
            before = []
            continue
        text = line.split("//")[0].strip()
        if not line.startswith("\t") or not text:
            continue
        if re.match(r"(global|buffer)_load_lds_", text):
            seen += 1
            m = re.search(r"s\[(\d+):(\d+)\]", text)
            base = set(range(int(m[1]), int(m[2]) + 1)) if m else set()
            waited = 0
            for p in reversed(before[-6:]):
                if waited < 1 and re.match(r"(s_\w+|v_readfirstlane_b32) m0\b", p):
                    early.append((p, text))
                w = re.match(r"v_read(?:first)?lane_b32 s(\d+)", p)
                if w and int(w[1]) in base and waited < 5:
                    early.append((p, text))
                nop = re.match(r"s_nop (\d+)", p)
                waited += int(nop[1]) + 1 if nop else 1
        before.append(text)
    return seen, early


def test_the_scan_finds_them():
    bad = ["0 <f>:", "\tv_readfirstlane_b32 s4, v1", "\ts_nop 0", "\ts_add_i32 m0, s1, 4",
           "\tglobal_load_lds_dwordx4 v2, s[4:5]"]
    assert len(hazards(bad)[1]) == 2
    good = bad[:4] + ["\ts_nop 4"] + bad[4:]
    assert hazards(good) == (1, [])


@pytest.mark.skipif(OBJDUMP is None, reason="no llvm-objdump")
def test_loads_to_lds_wait(tmp_path):
    if not os.path.exists(M.LIB_PATH):
        pytest.skip("library not built")
    seen, early = hazards(_disassembly(str(tmp_path)))
    assert seen > 100
    assert not early, early[:5]
