"""More of what test_matrix_waits_cpu.py looks for in the library's machine code: results of matrix
instructions that leave through other instructions than those it knows, and matrix instructions that multiply
one. Accumulation registers, which neither test follows, must not occur.

A matrix instruction that takes another's result as a factor needs the same wait states as a vector
instruction. One that adds to another's result needs none if it is that sum as a whole; a part of it counts as
any other use."""

import os
import re

import pytest

from test_matrix_waits_cpu import PASSES, functions, registers
from test_wait_states_cpu import LLVM_OBJDUMP, listings

# Whatever may read vector registers: vector and matrix instructions, LDS, and memory in all of its forms.
READERS = ("v_", "ds_", "flat_", "global_", "buffer_", "scratch_", "image_", "tbuffer_")


def vectors(operand):
    """An operand's vector registers; accumulation registers are none that this test knows."""
    assert not re.match(r"-?\|?a(\d+|\[)", operand), f"{operand}: accumulation registers are not followed"
    return registers(operand)


def early(code):
    """(matrix instruction, the instruction that touches its result too early, its wait states) along any path."""
    place = {at: i for i, (at, _, _, _) in enumerate(code)}
    found = []
    for i, (at, name, operands, _) in enumerate(code):
        need = PASSES.get(name)
        if need is None:
            assert not name.startswith(("v_mfma", "v_smfma")), f"{name}: its passes are not listed"
            continue
        result = vectors(operands[0])
        assert result, f"{name} {operands}: no result that is known"
        todo, best = [(i + 1, 0)], {}
        while todo:
            k, states = todo.pop()
            if k >= len(code) or states >= need or best.get(k, need) <= states:
                continue
            best[k] = states
            _, other, ops, target = code[k]
            if other.startswith("s_endpgm"):
                continue
            if other.startswith(READERS):
                touched = [vectors(o) & result for o in ops]
                if other.startswith("v_mfma") and vectors(ops[0]) == result and vectors(ops[3]) in (result, set()):
                    # the sum goes on, or the registers get another: that instruction's wait counts from here
                    if touched[1] or touched[2]:
                        found.append((at, f"{other} {' '.join(ops)}", states))
                    continue
                if any(touched):
                    found.append((at, f"{other} {' '.join(ops)}", states))
                    continue
            step = int(ops[0], 0) + 1 if other == "s_nop" else 1
            if target is not None:
                todo.append((place[target], states + step))
            if other != "s_branch":
                todo.append((k + 1, states + step))
    return found


PRODUCT = "v_mfma_f32_32x32x16_bf16 v[2:17], v[20:23], v[24:27], v[2:17]"


def found(*lines):
    listing = "0000000000000000 <k>:\n" + "".join(f"\t{t} // {4 * i:012X}: 00\n" for i, t in enumerate(lines))
    return len(early(functions(listing)["k"]))


@pytest.mark.parametrize("use", ["flat_store_dword v[40:41], v17", "scratch_store_dwordx4 off, v[14:17], s3", "global_atomic_add_f32 v40, v2, s[4:5]",
                                 "flat_atomic_add v[40:41], v9", "buffer_store_dword v5, v40, s[8:11], 0 offen", "ds_add_f32 v40, v3",
                                 "v_mfma_f32_32x32x16_bf16 v[44:59], v[14:17], v[24:27], v[44:59]",
                                 "v_mfma_f32_32x32x16_bf16 v[44:59], v[20:23], v[2:5], v[44:59]",
                                 "v_mfma_f32_32x32x16_bf16 v[2:17], v[20:23], v[2:5], v[2:17]",
                                 "v_mfma_f32_32x32x16_bf16 v[44:59], v[20:23], v[24:27], v[2:17]",
                                 "v_mfma_f32_32x32x16_bf16 v[10:25], v[60:63], v[64:67], v[10:25]", "v_mov_b32_e32 v30, v17"])
def test_the_check_sees(use):
    assert found(PRODUCT, use) == 1
    assert found(PRODUCT, "s_nop 7", "s_nop 1", use) == 1
    assert found(PRODUCT, "s_nop 7", "s_nop 2", use) == 0


def test_the_check_lets_sums_go_on():
    assert found(PRODUCT, PRODUCT, "v_mov_b32_e32 v30, v18") == 0
    assert found(PRODUCT, "v_mfma_f32_32x32x16_bf16 v[2:17], v[20:23], v[24:27], 0") == 0
    assert found(PRODUCT, "global_load_dwordx4 v[40:43], v44, s[4:5]") == 0


@pytest.mark.parametrize("lines", [("v_mfma_f32_32x32x16_bf16 a[0:15], v[20:23], v[24:27], a[0:15]",), (PRODUCT, "v_accvgpr_write_b32 a3, v17")])
def test_the_check_knows_no_accumulation_registers(lines):
    with pytest.raises(AssertionError, match="accumulation"):
        found(*lines)


@pytest.mark.skipif(not os.path.exists(LLVM_OBJDUMP), reason="no llvm-objdump")
def test_the_library(tmp_path):
    products, bad = 0, []
    for listing in listings(tmp_path):
        for name, code in functions(listing).items():
            products += sum(n in PASSES for _, n, _, _ in code)
            for _, n, ops, _ in code:
                assert not n.startswith("v_accvgpr"), f"{n} in {name}: accumulation registers are not followed"
            bad += [(name, *f) for f in early(code)]
    assert products > 0
    assert not bad, f"{len(bad)} results are touched too early, the first: {bad[0]}"
