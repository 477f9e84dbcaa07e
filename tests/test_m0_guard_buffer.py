"""The MX tiles' direct loads and the M0 register, checked on the built code.

They issue ``buffer_load_dwordx4 ... lds`` from inline assembly that first
moves the LDS destination into M0, which the compiler reserves for itself: in
every kernel with that sequence, M0 is written by it alone and nothing else
reads M0 (the other direct loads' rule, for the buffer form).
"""
from __future__ import annotations

import os
import re

import pytest

from test_m0_guard import BUILD, IMPLICIT_M0, MOV_M0, _tools_present, disassemble, instructions

BUFFER_LOAD = re.compile(r"^buffer_load_dwordx4 v\d+, s\[\d+:\d+\], (s\d+|0|vcc_lo|vcc_hi) offen lds$")


def _sequence(insts, i) -> bool:
    func = insts[i][0]
    return (i + 2 < len(insts) and bool(MOV_M0.match(insts[i][1])) and insts[i + 1] == (func, "s_nop 0")
            and insts[i + 2][0] == func and bool(BUFFER_LOAD.match(insts[i + 2][1])))


def violations(asm: str) -> tuple[int, list[str]]:
    insts = list(instructions(asm))
    starts = {i for i in range(len(insts)) if _sequence(insts, i)}
    funcs = {insts[i][0] for i in starts}
    bad = []
    for i, (func, text) in enumerate(insts):
        if func not in funcs:
            continue
        if re.search(r"\bm0\b", text) and i not in starts:
            bad.append(f"{func}: {text}")
        elif IMPLICIT_M0.match(text) and i - 2 not in starts:
            bad.append(f"{func}: {text}")
    return len(starts), bad


@pytest.mark.skipif(not _tools_present(), reason="binutils or the ROCm LLVM tools are missing")
def test_m0_used_only_by_buffer_direct_loads(tmp_path):
    obj = os.path.join(BUILD, "mx_gemm.o")
    if not os.path.exists(obj):
        pytest.skip("the library's objects are not built in this tree (run the build first)")
    count, bad = violations(disassemble(obj, str(tmp_path)))
    assert not bad, "\n".join(bad[:20])
    assert count > 100


def test_checker_catches_foreign_m0_uses():
    good = """
0000000000001000 <k>:
\ts_mov_b32 m0, s4
\ts_nop 0
\tbuffer_load_dwordx4 v1, s[8:11], s5 offen lds
\ts_endpgm
"""
    assert violations(good) == (1, [])
    assert violations(good.replace("\ts_endpgm", "\ts_mov_b32 m0, -1\n\ts_endpgm"))[1]
    assert violations(good.replace("\ts_endpgm", "\tbuffer_load_dwordx4 v1, s[8:11], s5 offen lds\n"
                                                 "\ts_endpgm"))[1]
    assert violations(good.replace("\ts_endpgm", "\tds_append v3\n\ts_endpgm"))[1]
