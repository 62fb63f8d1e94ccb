"""The distance that the 8-bit integer products keep between a matrix product and vector code that rewrites its operands.

tb_device.h (mfma_operand_guard) describes the form and the distance; the kernels of the integer product are read here
from the library that was built, along every path through their code: the rewrite of an operand may stand behind a
branch, or at the head of the loop.
"""

import glob
import os
import re
import shutil
import subprocess

import pytest

tb = pytest.importorskip("rank_factored_linear_amd.binding")

WAIT_STATES = 24
PRODUCT = "v_mfma_i32_16x16x64_i8"
OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump") or "") if os.path.exists(p)), None)


def _registers(operand):
    m = re.match(r"([va])\[(\d+):(\d+)\]|([va])(\d+)\b", operand)
    if not m:
        return set()
    return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)} if m[1] else {(m[4], int(m[5]))}


def kernels(code):
    """{kernel: [(address, instruction, operands, address of a branch's target)]} of disassembled code."""
    found, body, base = {}, None, 0
    for line in code.splitlines():
        head = re.match(r"([0-9a-f]+) <(.*)>:$", line)
        if head:
            base, body = int(head[1], 16), found.setdefault(head[2], [])
            continue
        m = re.match(r"\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+):(.*)$", line)
        if body is None or not m:
            continue
        target = None
        if m[1].startswith(("s_branch", "s_cbranch")):
            offset = re.search(r"<[^>]*?(?:\+0x([0-9a-f]+))?>", m[4])
            target = base + int(offset[1] or "0", 16)
        body.append((int(m[3], 16), m[1], re.findall(r"[vas]\[\d+:\d+\]|[vas]\d+\b|[^,\s]+", m[2]), target))
    return found


def rewrites(body):
    """([(product's address, vector instruction, wait states between them)], number of products): vector instructions
    that write an A or B register of a product fewer than WAIT_STATES behind it on some path.  An instruction counts as
    one wait state, s_nop n as n + 1."""
    at = {address: i for i, (address, *_) in enumerate(body)}
    bad, products = [], 0
    for i, (address, op, operands, _) in enumerate(body):
        if op != PRODUCT:
            continue
        products += 1
        held, least, paths = _registers(operands[1]) | _registers(operands[2]), {}, [(i + 1, 0)]
        while paths:
            j, states = paths.pop()
            if j >= len(body) or states >= least.get(j, WAIT_STATES):
                continue
            least[j] = states
            _, op, operands, target = body[j]
            if op.startswith("v_") and not op.startswith(("v_mfma", "v_cmp")):
                written = _registers(operands[0]) | (_registers(operands[1]) if op.startswith("v_swap") else set())
                if written & held:
                    bad.append((hex(address), f"{op} {' '.join(operands)}", states))
            states += int(operands[0], 0) + 1 if op == "s_nop" else 1
            if target is not None:
                paths.append((at[target], states))
            if op not in ("s_endpgm", "s_branch"):
                paths.append((j + 1, states))
    return bad, products


def test_the_scan_follows_branches():
    code = """0000000000000100 <k>:
	v_mov_b32_e32 v4, 0                  // 000000000100: 00000000
	s_nop 7                              // 000000000104: 00000000
	v_mfma_i32_16x16x64_i8 v[0:3], v[4:7], v[8:11], v[0:3]  // 000000000108: 00000000 00000000
	s_nop 7                              // 000000000110: 00000000
	s_cbranch_scc1 2                     // 000000000114: 00000000 <k+0x20>
	s_nop 4                              // 000000000118: 00000000
	v_cmp_eq_u32_e32 vcc, v4, v5         // 00000000011C: 00000000
	v_mov_b32_e32 v9, 0                  // 000000000120: 00000000
	v_mov_b32_e32 v0, 0                  // 000000000124: 00000000
	s_cbranch_scc0 65533                 // 000000000128: 00000000 <k>
	s_endpgm                             // 00000000012C: 00000000
"""
    bad, products = rewrites(kernels(code)["k"])
    assert products == 1
    least = {}
    for _, text, states in bad:
        register = text.split()[1]
        least[register] = min(states, least.get(register, states))
    # v9 by the branch that is taken; v4 round the loop; v0 is a result.
    assert least == {"v9": 9, "v4": 12}


@pytest.mark.skipif(OBJDUMP is None, reason="no llvm-objdump")
def test_operands_of_integer_products_outlive_them(tmp_path):
    shutil.copy(tb.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, stdout=subprocess.DEVNULL)
    checked = {"decode": 0, "ring": 0, "tiles": 0}
    for image in sorted(glob.glob(str(tmp_path / "lib.so.*gfx950"))):
        code = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", image], check=True, capture_output=True, text=True).stdout
        if PRODUCT not in code:
            continue
        for name, body in kernels(code).items():
            bad, products = rewrites(body)
            assert not bad, (name, len(bad), sorted(bad, key=lambda b: b[2])[:4])
            if products:
                checked[re.search("int8_(decode|ring|tiles)_kernel", name)[1]] += 1
    assert checked == {"decode": 44, "ring": 6, "tiles": 2}
