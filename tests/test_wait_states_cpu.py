"""The wait states that gfx950's buffer loads need before them, in the library's
machine code. The compiler puts them in where it emits both instructions
itself, but not inside inline assembly:

- a direct load to LDS reads M0, which must not have been written by the
  instruction just before it;
- a buffer instruction must not read a scalar register that a vector
  instruction wrote less than five instructions before.
"""

import glob
import os
import re
import shutil
import subprocess

import pytest

rar = pytest.importorskip("ring_all_reduce_ddp_amd")

LLVM_OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def scalars(operand):
    """The scalar registers of an operand: s5, s[4:7]."""
    m = re.fullmatch(r"s(\d+)", operand)
    if m:
        return {int(m.group(1))}
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    return set(range(int(m.group(1)), int(m.group(2)) + 1)) if m else set()


def faults(listing):
    """(kernel, what, instruction) of every buffer load that comes too early."""
    out, kernel, recent = [], None, []   # recent: (writes M0, scalars a vector instruction wrote), newest last
    for line in listing.splitlines():
        head = re.fullmatch(r"[0-9a-f]+ <(.+)>:", line)
        if head:
            kernel, recent = head.group(1), []
            continue
        text = line.split("//")[0].strip()
        if not line.startswith("\t") or not text:
            continue
        name, _, rest = text.partition(" ")
        operands = [o for o in re.split(r"[ ,]+", rest) if o]
        if name == "s_nop":
            recent += [(False, set())] * (int(operands[0], 0) + 1)
            continue
        if name.startswith(("buffer_", "global_", "scratch_")):
            to_lds = "lds" in operands or "_lds_" in name
            if to_lds and recent and recent[-1][0]:
                out.append((kernel, "M0", text))
            read = set().union(*(scalars(o) for o in operands))
            if any(read & wrote for _, wrote in recent[-5:]):
                out.append((kernel, "scalar", text))
        first = operands[0] if operands else ""
        recent.append((first == "m0", scalars(first) if name.startswith("v_") else set()))
    return out


def listings(tmp_path):
    """Disassembly of each code object in the library built here."""
    copy = os.path.join(tmp_path, "lib.so")
    shutil.copy(rar.LIB_PATH, copy)
    subprocess.run([LLVM_OBJDUMP, "--offloading", copy], check=True, stdout=subprocess.DEVNULL, cwd=tmp_path)
    objects = sorted(glob.glob(copy + "*gfx950"))
    assert objects, "the library has no gfx950 code"
    for o in objects:
        yield subprocess.run([LLVM_OBJDUMP, "-d", o], check=True, stdout=subprocess.PIPE, text=True).stdout


def test_the_check_sees_missing_wait_states():
    def found(*lines):
        return [what for _, what, _ in faults("0000 <k>:\n" + "".join(f"\t{t}   // 00: 00\n" for t in lines))]
    load = "buffer_load_dwordx4 v6, s[8:11], 0 offen lds"
    assert found("s_mov_b32 m0, s33", load) == ["M0"]
    assert found("s_mov_b32 m0, s33", "s_nop 0", load) == []
    assert found("s_mov_b32 m0, s33", "v_mov_b32_e32 v1, v2", load) == []
    assert found("v_readfirstlane_b32 s9, v1", "s_nop 3", load) == ["scalar"]
    assert found("v_readfirstlane_b32 s9, v1", "s_nop 4", load) == []
    assert found("v_readfirstlane_b32 s12, v1", load) == []
    assert found("v_cmp_gt_i32_e64 s[10:11], s15, v156", load) == ["scalar"]


@pytest.mark.skipif(not os.path.exists(LLVM_OBJDUMP), reason="no llvm-objdump")
def test_buffer_loads_wait_for_their_scalars(tmp_path):
    loads = 0
    for listing in listings(tmp_path):
        loads += len(re.findall(r"\boffen lds\b", listing))
        bad = faults(listing)
        assert not bad, f"{len(bad)} loads come too early, the first: {bad[0]}"
    assert loads > 0
