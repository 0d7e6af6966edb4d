"""Inline-assembly loads wait for their scalar operands.  A vector instruction that writes a
scalar register (v_readfirstlane, a compare, the restore of a spilled register) must be five
wait states ahead of a memory instruction that reads it; the compiler sees to that for its
own instructions, but not for those inside an asm statement, so the statement has to begin
with the wait."""
import pathlib
import re

import pytest

from test_asm_clobbers import CSRC, _asm_statements

_LOAD = re.compile(r"\b(buffer|global)_(load|store|atomic)\w*")


def wait_states(template):
    """Wait states of a statement ahead of its first memory instruction, None without one."""
    states = 0
    for line in re.split(r"\\n", template):
        line = line.replace("\\t", "").strip()
        if not line:
            continue
        if _LOAD.match(line):
            return states
        nop = re.match(r"s_nop (\d+)", line)
        states += 1 + (int(nop.group(1)) if nop else 0)
    return None


@pytest.mark.parametrize("name", ["ssd_mma.h", "ssd_paged.hip", "ssd_paged_rows.hip", "ssd_attn.hip", "ssd_linattn.hip"])
def test_loads_wait_for_scalar_operands(name):
    for line, template, _ in _asm_statements((CSRC / name).read_text()):
        states = wait_states(template)
        assert states is None or states >= 5, f"{name}:{line}: {states} wait states ahead of the load"


def test_the_scan_finds_what_it_should():
    assert wait_states(r"s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds") == 2
    assert wait_states(r"s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dword %1, %2") == 6
    assert wait_states(r"s_waitcnt vmcnt(%0)") is None
