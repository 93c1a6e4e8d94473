"""The wide attention kernels chain matrix products in assembly statements,
for which the compiler counts no wait states: nothing may touch a chain's sum
between its products, nor within the wait states that its last product
carries.  Read from the assembly that hipcc writes for csrc/mla_decode.hip
(compiled here for gfx950; no GPU)."""

import os
import re
import shutil
import subprocess

import pytest

from mxfp4_block_scaled_quant_amd import build as B

SOURCE = os.path.join(B.CSRC, "mla_decode.hip")
SETTLED = 19  # wait states from an 8-pass matrix product to its result's use, and some to spare


def registers(operand):
    m = re.fullmatch(r"v\[(\d+):(\d+)\]", operand) or re.fullmatch(r"v(\d+)()", operand)
    return set(range(int(m.group(1)), int(m.group(2) or m.group(1)) + 1)) if m else set()


def chain_faults(lines):
    """(products in chains, lines that break the rule)."""
    products, faults, pending, waited, inside = 0, [], set(), 0, False
    for line in map(str.strip, lines):
        if line.startswith(";;#ASM"):
            inside = line.startswith(";;#ASMSTART")
            continue
        if not line or line[0] in ";." or line.endswith(":"):
            continue
        op, *rest = line.split()
        operands = [x.strip(",") for x in rest]
        if inside and op.startswith("v_mfma"):
            products += 1
            sums = registers(operands[0])
            sources = registers(operands[1]) | registers(operands[2])
            if pending and (sources & pending or (operands[3] != "0" and sums != pending)):
                faults.append(line)
            pending, waited = sums, 0
        elif op == "s_nop":
            waited += int(operands[0]) + 1
            if waited >= SETTLED:
                pending = set()
        elif pending and any(registers(x) & pending for x in operands):
            faults.append(line)
    return products, faults


def test_the_reader_finds_a_copy_inside_a_chain():
    chain = [";;#ASMSTART", "v_mfma_f32_32x32x16_bf16 v[2:17], v[20:23], v[24:27], 0", ";;#ASMEND"]
    more = [";;#ASMSTART", "v_mfma_f32_32x32x16_bf16 v[2:17], v[28:31], v[24:27], v[2:17]", ";;#ASMEND"]
    assert chain_faults(chain + ["v_add_f32_e32 v30, v31, v32"] + more) == (2, [])
    assert chain_faults(chain + ["v_mov_b64_e32 v[40:41], v[2:3]"] + more)[1]
    moved = [x.replace("v[2:17]", "v[40:55]") for x in more]
    assert chain_faults(chain + moved)[1]
    assert chain_faults(chain + ["s_nop 3", "v_mov_b32_e32 v40, v5"])[1]
    assert not chain_faults(chain + ["s_nop 15", "s_nop 3", "v_mov_b32_e32 v40, v5"])[1]


@pytest.mark.skipif(not (os.path.exists(B.HIPCC) or shutil.which(B.HIPCC)), reason="needs hipcc")
def test_no_instruction_touches_a_chain(tmp_path):
    out = str(tmp_path / "mla_decode.s")
    flags = [*B.FLAGS, *B.FILE_FLAGS.get("mla_decode.hip", [])]
    r = subprocess.run([B.HIPCC, *flags, "--cuda-device-only", "-S", SOURCE, "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    products, faults = chain_faults(open(out).read().split("\n"))
    assert products and products % 36 == 0     # 36 products a chain
    assert not faults, faults[:5]
