"""Forms that the device compiler gets wrong, kept out of the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "laplacian_nystr_linear_gb300", "csrc")


def bare_loops(s):
    """Lines of an `if constexpr`, or its else, whose substatement is a loop without braces around it.  nvcc 13.0.88
    drops the statement behind such a loop, where it is discarded, in a lambda of a function template."""
    found = []
    for m in re.finditer(r"\bif constexpr\s*\(", s):
        i, deep = m.end(), 1
        while deep:
            deep += (s[i] == "(") - (s[i] == ")")
            i += 1
        blank = r"(?:\s|//[^\n]*\n|#pragma[^\n]*\n)*"
        if re.match(blank + r"(for|while|do)\b", s[i:]):
            found.append(s.count("\n", 0, m.start()) + 1)
        # the else of a one-line substatement or of a block that ends there
        rest = re.match(blank + r"(?:[^;{}]*;|\{[^{}]*\})" + blank + r"else" + blank + r"(for|while|do)\b", s[i:])
        if rest:
            found.append(s.count("\n", 0, m.start()) + 1)
    return found


def test_the_search_finds_them():
    assert bare_loops("if constexpr (A(1))  // b\n#pragma unroll\n for (;;) { x(); }") == [1]
    assert bare_loops("\nif constexpr (A) x = 1;\n else\n while (y) { x(); }") == [2]
    assert bare_loops("if constexpr (A) {\n for (;;) { x(); } } else if constexpr (B) { y(); }") == []


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_no_bare_loop_behind_if_constexpr(path):
    with open(path) as f:
        assert bare_loops(f.read()) == []
