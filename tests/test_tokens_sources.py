"""What the sources of libdlrm_tokens.so keep to, where no run would show it for certain."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOKENS = os.path.join(ROOT, "dlrm_embedding_bag_b200", "csrc", "tokens")
SOURCES = sorted(glob.glob(os.path.join(TOKENS, "*.cu")) + glob.glob(os.path.join(TOKENS, "*.h")))


def _code(path):
    """A source without its comments."""
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def _asm_statements(code):
    for m in re.finditer(r"\basm\b\s*(volatile)?\s*\(", code):
        i, depth = m.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(code[i], 0)
            i += 1
        yield m.group(1) is not None, code[m.end():i - 1]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_memory_accesses_in_assembly_stay_where_they_are_written(path):
    """An access in inline assembly is volatile and names memory: else the compiler may
    move it over a wait or a barrier."""
    for volatile, text in _asm_statements(_code(path)):
        first = re.match(r'[\s"{\\nt]*([a-z]+[\w.:]*)', text).group(1)
        if re.match(r"(ld|st|cp|red|atom|mbarrier|griddepcontrol|barrier|bar|fence)\b", first):
            assert volatile, text
            if not re.match(r"(ld|st)\.(param|const)", first):
                assert '"memory"' in text, text


def test_kernels_that_start_early_read_nothing_through_the_read_only_path():
    """The layer is scheduled while the kernel in front of it, which may write any of its
    operands, is at work: read-only loads could be moved in front of its wait, and are not
    coherent with writes of the time that it has run."""
    code = _code(os.path.join(TOKENS, "linear_int8.cu"))
    assert code.count("griddepcontrol.wait") == 2
    assert "__ldg" not in code and ".nc" not in code
    # the gradient's kernels that start early read only what no kernel writes meanwhile:
    # ids (final before the first launch of the sort, which does not start early)
    code = _code(os.path.join(TOKENS, "embedding.cu"))
    kernels = re.split(r"\n__global__", code)[1:]
    early = [k[:k.index("\n}\n")] for k in kernels if "griddepcontrol.wait" in k[:k.index("\n}\n")]]
    assert len(early) >= 4
    for k in early:
        assert "__ldg" not in k


def test_tensor_memory_loads_are_waited_for_in_their_own_statement():
    """Registers that a tcgen05.ld fills arrive with its wait: no statement may come between."""
    found = 0
    for path in glob.glob(os.path.join(os.path.dirname(TOKENS), "*.cu*")) + SOURCES:
        for volatile, text in _asm_statements(_code(path)):
            if "tcgen05.ld." in text:
                found += 1
                assert volatile and "tcgen05.wait::ld" in text and '"memory"' in text, path
            else:
                assert "tcgen05.wait::ld" not in text, path
    assert found >= 1
