"""What the sources of libdlrm_narrow.so keep to, where no run would show it for certain."""
import glob
import os
import re

import pytest

from test_tokens_sources import ROOT, _asm_statements, _code

NARROW = os.path.join(ROOT, "dlrm_embedding_bag_b200", "csrc", "narrow")
SOURCES = sorted(glob.glob(os.path.join(NARROW, "*.cu*")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_memory_accesses_in_assembly_stay_where_they_are_written(path):
    """An access in inline assembly is volatile and names memory: else the compiler may
    move it over a wait or a barrier."""
    for volatile, text in _asm_statements(_code(path)):
        first = re.match(r'[\s"{\\nt]*([a-z]+[\w.:]*)', text).group(1)
        if re.match(r"(ld|st|cp|red|atom|mbarrier|griddepcontrol|barrier|bar|fence)\b", first) or \
                re.match(r"tcgen05\.(ld|st|cp|wait|mma|commit)", text.strip(' "\n')):
            assert volatile and '"memory"' in text, text


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_nothing_is_read_through_the_read_only_path(path):
    """Kernels start while the one in front of them, which may write any of their operands, is
    at work; the optimiser's writes what it reads."""
    code = _code(path)
    assert "__ldg" not in code and ".nc" not in code


def test_kernels_that_start_early_wait_first():
    """Every kernel but the optimiser's, which do not start early, waits for the one in front of it
    before any access; none lets the next one start before its own end."""
    for path in SOURCES:
        code = _code(path)
        assert "launch_dependents" not in code
        for body in re.split(r"\n__global__", code)[1:]:
            body = body[:body.index("\n}\n")]
            assert ("griddepcontrol.wait" in body) == (os.path.basename(path) != "adamw.cu"), path
    early = "".join(_code(p) for p in SOURCES if p.endswith("adamw.cu"))
    assert not re.search(r"kThreads, 0, true|256, 0, true", early)


def test_tensor_memory_stores_are_waited_for():
    """What a warp wrote to tensor memory has arrived before it says so."""
    code = _code(os.path.join(NARROW, "linear_fp4.cu"))
    at = code.index("tmem_st_8(to")
    assert re.match(r"tmem_st_8\(to \+ i, r \+ i\);\s*tmem_st_wait\(\);\s*arrive\(", code[at:])
    assert code.count("tcgen05.ld.") == 0  # loads are those of the shared header, waited for there
