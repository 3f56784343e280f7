"""Results of matrix instructions in the library's machine code: nothing but
another matrix instruction may touch them before the hardware has written them,
which takes as many wait states as a compiler has to put in. It has been seen to
leave some out where a branch leads from the instruction straight to the copies
of its results, so every path is followed here.

Wait states before a vector instruction, a store or an LDS write that touches
the result: 11 after an instruction of 8 passes (32 x 32 x 16 of bf16), 18 after one
of 16 (32 x 32 x 2 of fp32). An instruction counts as one, s_nop n as n + 1."""

import os
import re

import pytest

from test_wait_states_cpu import LLVM_OBJDUMP, listings

PASSES = {"v_mfma_f32_32x32x16_bf16": 11, "v_mfma_f32_32x32x2_f32": 18, "v_mfma_f32_32x32x2f32": 18}


def registers(operand):
    m = re.fullmatch(r"-?\|?v(\d+)\|?", operand)
    if m:
        return {int(m.group(1))}
    m = re.fullmatch(r"v\[(\d+):(\d+)\]", operand)
    return set(range(int(m.group(1)), int(m.group(2)) + 1)) if m else set()


def functions(listing):
    """{name: [(address, mnemonic, operands, branch target or None)]}"""
    out, current = {}, None
    for line in listing.splitlines():
        head = re.fullmatch(r"([0-9a-f]+) <(.+)>:", line)
        if head:
            current = out.setdefault(head.group(2), [])
            start = int(head.group(1), 16)
            continue
        m = re.match(r"\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):", line)
        if not m or current is None:
            continue
        name, rest, at = m.group(1), m.group(2), int(m.group(3), 16)
        target = None
        if name.startswith(("s_branch", "s_cbranch")):
            t = re.search(r"<.*?(?:\+0x([0-9a-fA-F]+))?>\s*$", line)
            target = start + (int(t.group(1), 16) if t and t.group(1) else 0)
        current.append((at, name, [o for o in re.split(r"[ ,]+", rest) if o], target))
    return out


def early(code):
    """(matrix instruction, the instruction that comes too early, its wait states) along any path."""
    place = {at: i for i, (at, _, _, _) in enumerate(code)}
    found = []
    for i, (at, name, operands, _) in enumerate(code):
        need = PASSES.get(name)
        if need is None:
            assert not name.startswith("v_mfma"), f"{name}: its passes are not listed"
            continue
        result = registers(operands[0])
        todo, best = [(i + 1, 0)], {}
        while todo:
            k, states = todo.pop()
            if k >= len(code) or states >= need or best.get(k, need) <= states:
                continue
            best[k] = states
            _, other, ops, target = code[k]
            if other.startswith("s_endpgm"):
                continue
            if other.startswith("v_mfma"):
                if registers(ops[0]) & result and registers(ops[0]) != result:
                    found.append((at, other, states))
                if registers(ops[0]) == result:
                    continue   # the sum goes on: that instruction's wait counts
            elif other.startswith(("v_", "ds_write", "global_store", "buffer_store", "ds_bpermute")) and \
                    any(registers(o) & result for o in ops):
                found.append((at, f"{other} {' '.join(ops)}", states))
                continue
            step = int(ops[0], 0) + 1 if other == "s_nop" else 1
            if target is not None:
                todo.append((place[target], states + step))
            if other != "s_branch":
                todo.append((k + 1, states + step))
    return found


def test_the_check_sees_a_result_read_too_early():
    def found(*lines):
        listing = "0000000000000000 <k>:\n" + "".join(f"\t{t} // {4 * i:012X}: 00{b}\n" for i, (t, b) in enumerate(lines))
        return len(early(functions(listing)["k"]))
    product = ("v_mfma_f32_32x32x16_bf16 v[2:17], v[20:23], v[24:27], v[2:17]", "")
    assert found(product, ("v_mov_b32_e32 v30, v17", "")) == 1
    assert found(product, ("s_nop 7", ""), ("s_nop 2", ""), ("v_mov_b32_e32 v30, v17", "")) == 0
    assert found(product, ("s_nop 7", ""), ("s_nop 1", ""), ("v_mov_b32_e32 v30, v17", "")) == 1
    assert found(product, ("v_mov_b32_e32 v30, v18", "")) == 0
    assert found(product, product, ("ds_write_b128 v40, v[14:17]", "")) == 1
    # a branch over the instructions that would have waited
    assert found(product, ("s_cbranch_vccz 3", " <k+0x10>"), ("s_nop 7", ""), ("s_nop 7", ""), ("v_mov_b64_e32 v[30:31], v[16:17]", "")) == 1


@pytest.mark.skipif(not os.path.exists(LLVM_OBJDUMP), reason="no llvm-objdump")
def test_matrix_results_are_not_read_too_early(tmp_path):
    products, bad = 0, []
    for listing in listings(tmp_path):
        for name, code in functions(listing).items():
            products += sum(n in PASSES for _, n, _, _ in code)
            bad += [(name, *f) for f in early(code)]
    assert products > 0
    assert not bad, f"{len(bad)} results are read too early, the first: {bad[0]}"
