"""The built library's own code, where the compiler cannot keep a rule of the machine
for what stands in inline asm: exchanges between lanes (permlane swaps, DPP) read no
register that one of the two vector instructions before them wrote, and results of the
transcendental unit are not read by the very next one.  A wait state is an instruction,
or one of an s_nop."""
import os
import re
import shutil
import subprocess

import pytest

import dequant_gemv_qgemv_amd as q
from dequant_gemv_qgemv_amd import _build

OBJDUMP = os.path.join(os.path.dirname(os.path.realpath(_build.HIPCC)), "..", "lib", "llvm", "bin", "llvm-objdump")
TRANSCENDENTAL = re.compile(r"v_(exp|log|rcp|rsq|sqrt|sin|cos|rcp_iflag)_")


def registers(operand):
    m = re.search(r"\bv(\d+)\b", operand)
    if m:
        return {int(m.group(1))}
    m = re.search(r"\bv\[(\d+):(\d+)\]", operand)
    return set(range(int(m.group(1)), int(m.group(2)) + 1)) if m else set()


def too_close(lines):
    """Lines that read a vector register too soon after the line that wrote it."""
    found, exchanges, recent = [], 0, []  # recent: (registers written, wait states since, transcendental)
    for line in lines:
        if line.endswith(">:"):
            recent = []
            continue
        text = line.split("//")[0].strip()
        if not text or text.startswith("Disassembly"):
            continue
        name, _, rest = text.partition(" ")
        operands = rest.split(",")
        swap = name.startswith("v_permlane")
        dpp = "row_" in rest or "quad_perm" in rest
        vector = name.startswith("v_")
        read = set().union(*map(registers, operands if swap else operands[1:])) if vector else set()
        exchanges += swap or dpp
        for written, since, slow in recent:
            need = 2 if swap else 1 if slow and not TRANSCENDENTAL.match(name) else 0
            if dpp:  # only the operand that is exchanged is read early
                need = 2 if written & registers(operands[1]) else need
            if vector and since < need and written & read:
                found.append((text, since))
        step = int(operands[0], 0) + 1 if name == "s_nop" else 1
        recent = [(w, s + step, t) for w, s, t in recent if s + step < 2]
        if vector and not name.startswith(("v_cmp", "v_readlane", "v_readfirstlane", "v_mfma")):
            recent.append((registers(operands[0]) | (registers(operands[1]) if swap or name.startswith("v_swap") else set()), 0,
                           bool(TRANSCENDENTAL.match(name))))
    return found, exchanges


def test_the_scan_itself():
    assert too_close(["v_max_f32_e32 v3, v1, v2", "v_permlane16_swap_b32_e32 v4, v3"])[0]
    assert too_close(["v_max_f32_e32 v3, v1, v2", "v_mov_b32_e32 v9, 0", "v_permlane32_swap_b32_e32 v3, v4"])[0]
    assert not too_close(["v_max_f32_e32 v3, v1, v2", "s_nop 1", "v_permlane32_swap_b32_e32 v3, v4"])[0]
    assert not too_close(["v_max_f32_e32 v3, v1, v2", "v_permlane32_swap_b32_e32 v5, v4"])[0]
    assert too_close(["v_permlane32_swap_b32_e32 v5, v4", "v_mov_b32_dpp v1, v4 row_ror:8 row_mask:0xf bank_mask:0xf"])[0]
    assert not too_close(["v_mov_b32_e32 v1, 0", "v_mov_b32_dpp v1, v4 row_ror:8 row_mask:0xf bank_mask:0xf"])[0]
    assert too_close(["v_exp_f32_e32 v1, v2", "v_add_f32_e32 v3, v1, v2"])[0]
    assert not too_close(["v_exp_f32_e32 v1, v2", "s_nop 0", "v_add_f32_e32 v3, v1, v2"])[0]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_waits_of_exchanges_between_lanes(tmp_path):
    shutil.copy(q.library_path(), tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    parts = sorted(f for f in os.listdir(tmp_path) if "gfx950" in f)
    assert len(parts) == len(_build.UNITS)
    total = 0
    for part in parts:
        text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", "--no-show-raw-insn", part], cwd=tmp_path, check=True, capture_output=True,
                              text=True).stdout
        found, exchanges = too_close(text.splitlines())
        assert not found, (part, found[:5])
        total += exchanges
    assert total > 500
