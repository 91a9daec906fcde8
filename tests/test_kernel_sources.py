"""What inline assembly in the kernels must leave to the compiler.

The compiler adds the software wait states of gfx950 where it issues the
instructions itself; inside inline assembly it sees none of them."""

import glob
import os
import re

import pytest

pytestmark = pytest.mark.cpu

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "manifold_constrained_hyper_amd",
                    "csrc")


def _asm_statements():
    """(file, template, rest) of every inline assembly statement: its text, and
    its operands and clobbers."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", code):
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(code[end], 0)
                end += 1
            template, _, rest = code[m.end():end - 1].partition(":")
            found.append((os.path.basename(path), template, rest))
    return found


def test_statements_are_found():
    """The reader of the sources sees the statements it is to judge."""
    texts = [t for _, t, _ in _asm_statements()]
    assert any("s_barrier" in t for t in texts) and any("global_load_lds" in t for t in texts)


def test_wait_state_between_m0_and_direct_to_lds_loads():
    """A direct-to-LDS load takes its LDS address from M0, which has to be
    written one wait state earlier (CDNA3 ISA, manually inserted wait states:
    S_MOV to M0, then a global load with LDS = 1)."""
    seen = 0
    for f, template, _ in _asm_statements():
        lines = [t.strip() for t in re.sub(r"[\"\n]", "", template).replace("\\t", " ").split("\\n")]
        for a, b in zip(lines, lines[1:]):
            if re.match(r"s_\w+ m0\b", a):
                seen += 1
                assert b.startswith("s_nop"), (f, template)
        assert not re.match(r"s_\w+ m0\b", lines[-1]), (f, template)
    assert seen


def test_no_dot_or_matrix_product_in_inline_assembly():
    """Another vector instruction may read a dot product's result only three
    wait states later, and a matrix product's later still."""
    bad = [(f, t) for f, t, _ in _asm_statements() if re.search(r"\bv_(dot|s?mfma|smfmac|wmma)", t)]
    assert not bad, bad


def test_asm_that_writes_m0_says_so():
    """M0 is also what the compiler's own direct-to-LDS loads and lane moves
    by M0 read: it has to know that its value is gone."""
    seen = 0
    for f, template, rest in _asm_statements():
        if re.search(r"\bs_\w+ m0\b", template):
            seen += 1
            assert '"m0"' in rest, (f, template)
    assert seen
