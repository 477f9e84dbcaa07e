"""The row tiles' and adapters' direct loads and the M0 register, checked on the built
code: the rule of test_m0_guard_buffer.py for the experts' and the adapters' kernels."""
from __future__ import annotations

import os

import pytest

from test_m0_guard import BUILD, _tools_present, disassemble
from test_m0_guard_buffer import violations


@pytest.mark.skipif(not _tools_present(), reason="binutils or the ROCm LLVM tools are missing")
@pytest.mark.parametrize("unit", ["experts_up", "experts_down", "experts_du", "experts_dw", "adapters", "adapters_thin"])
def test_m0_used_only_by_buffer_direct_loads(tmp_path, unit):
    obj = os.path.join(BUILD, unit + ".o")
    if not os.path.exists(obj):
        pytest.skip("the library's objects are not built in this tree (run the build first)")
    count, bad = violations(disassemble(obj, str(tmp_path)))
    assert not bad, "\n".join(bad[:20])
    assert count > 50
