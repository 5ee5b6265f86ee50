"""The hand-written loads to LDS of the 8-bit head's product, in the assembly that the library's own flags give (CPU:
hipcc cross-compiles).

Their base address stands in scalar registers.  A vector instruction that writes a scalar register (a lane read, a
comparison, a carry) needs 5 wait states before a memory instruction may read it; the compiler inserts them for its own
loads, but not for one inside inline assembly.  So no such write may come that close in front of one.
"""

import os
import re
import shutil
import subprocess

import pytest

from draft_verification_04_amd import build as B

FLAGS = [f for f in B.FLAGS if f not in ("-fPIC", "-shared")] + ["--cuda-device-only", "-S"]
WAIT_STATES = 5


def _scalars(text):
    """The scalar registers that an operand list names."""
    regs = set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        regs.update(range(int(a), int(b) + 1))
    regs.update(int(a) for a in re.findall(r"\bs(\d+)\b", text))
    return regs


def _instructions(asm):
    out = []
    for line in asm.splitlines():
        line = re.split(r";|//", line)[0].strip()
        if re.match(r"[a-z]\w*(\s|$)", line) and not line.endswith(":"):
            op, _, rest = line.partition(" ")
            op, _, more = op.partition("\t")
            out.append((op, (more + " " + rest).strip()))
    return out


def _written_by_vector(op, operands):
    """Scalar registers among the instruction's destinations: the first operand, the second one, too, of a carry."""
    if not op.startswith("v_"):
        return set()
    parts = [p.strip() for p in operands.split(",")]
    return _scalars(parts[0]) | (_scalars(parts[1]) if "_co_" in op or "div_scale" in op or "mad_u64" in op or
                                 "mad_i64" in op else set())


def _too_close(instructions):
    bad, loads = [], 0
    for n, (op, operands) in enumerate(instructions):
        if not op.startswith("global_load_lds"):
            continue
        loads += 1
        base, states = _scalars(operands), 0
        assert len(base) == 2, (op, operands)
        for k in range(n - 1, -1, -1):
            before, what = instructions[k]
            if states >= WAIT_STATES:
                break
            if _written_by_vector(before, what) & base:
                bad.append((before, what, op, operands))
            states += int(what, 0) + 1 if before == "s_nop" else 1
    return loads, bad


def test_the_check_sees_what_it_looks_for():
    asm = "\tv_readfirstlane_b32 s5, v1\n\ts_mov_b32 m0, s9\n\ts_nop 0\n\tglobal_load_lds_dwordx4 v0, s[4:5]\n"
    assert len(_too_close(_instructions(asm))[1]) == 1
    assert _too_close(_instructions(asm.replace("s_nop 0", "s_nop 4"))) == (1, [])
    assert _too_close(_instructions(asm.replace("s5", "s6"))) == (1, [])
    assert len(_too_close(_instructions(asm.replace("v_readfirstlane_b32 s5, v1", "v_add_co_u32 v1, s[4:5], v2, v3")))[1]) == 1


def test_bases_come_from_the_scalar_unit(tmp_path):
    if not os.path.exists(B.HIPCC) and shutil.which("hipcc") is None:
        pytest.skip("hipcc not found")
    out = str(tmp_path / "logits.s")
    subprocess.run([B.HIPCC] + FLAGS + ["-I", B.INCLUDE, "-I", B.CSRC, os.path.join(B.CSRC, "logits.hip"), "-o", out], check=True,
                   capture_output=True, timeout=600)
    with open(out) as f:
        loads, bad = _too_close(_instructions(f.read()))
    assert loads > 100 and not bad, (loads, bad[:5])
