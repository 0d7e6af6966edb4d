"""Direct loads into LDS, which the sources write as asm statements, keep the distances that the
hardware does not see to and the compiler does not either inside such a statement: five wait
states between a vector instruction that writes a scalar register, which may be the last one
ahead of the statement, and a memory instruction that reads it, and one between writing m0 and
a load into LDS.  Every source and header of the library is read."""
import re

import pytest

from test_asm_clobbers import _asm_statements, _sources
from test_asm_wait_states import wait_states

_DIRECT = re.compile(r"\b(buffer|global)_load_\w+.*(\blds\b|_lds_)|\bglobal_load_lds_\w+")


def instructions(template):
    return [x for x in (y.replace("\\t", "").strip() for y in re.split(r"\\n", template)) if x]


def is_direct(template):
    return any(_DIRECT.search(x) for x in instructions(template))


def after_m0(template):
    """Wait states between the statement's last write of m0 and its first load into LDS (None
    without such a load or where nothing of the statement writes m0)."""
    states = None
    for line in instructions(template):
        if _DIRECT.search(line):
            return states
        nop = re.match(r"s_nop (\d+)", line)
        if re.match(r"s_\w+ m0,", line):
            states = 0
        elif states is not None:
            states += 1 + (int(nop.group(1)) if nop else 0)
    return None


def direct_loads(path):
    return [(line, t) for line, t, _ in _asm_statements(path.read_text()) if is_direct(t)]


@pytest.mark.parametrize("path", _sources(), ids=lambda p: p.name)
def test_statements_keep_their_distances(path):
    for line, template, _ in _asm_statements(path.read_text()):
        states = wait_states(template)
        assert states is None or states >= 5, f"{path.name}:{line}: {states} wait states ahead of a memory instruction"
        if is_direct(template):
            m0 = after_m0(template)
            assert m0 is not None and m0 >= 1, f"{path.name}:{line}: {m0} wait states between m0 and the load"


def test_all_direct_loads_are_found():
    """The bf16 scan's two, the shared one and the 4-bit pages' two."""
    found = {p.name: len(direct_loads(p)) for p in _sources()}
    assert {n: c for n, c in found.items() if c} == {"ssd_scan_bf16.hip": 2, "ssd_mma.h": 1, "ssd_paged.hip": 2}


def test_the_reader_counts_as_the_hardware_does():
    assert after_m0(r"s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds") == 0
    assert after_m0(r"s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2") == 1
    assert after_m0(r"s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds") == 5
    assert after_m0(r"buffer_load_dwordx4 %1, %2, %3 offen") is None
