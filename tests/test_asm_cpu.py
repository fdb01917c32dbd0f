"""Inline assembly in csrc/: a statement that writes m0 names it as clobbered, so
that the compiler keeps nothing of its own there across it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_verify_gdn_amd", "csrc")


def statements(text):
    """The asm statements of a source, each up to its closing parenthesis."""
    for m in re.finditer(r"\basm\b\s*(?:volatile\b\s*)?\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if quoted:
                i += c == "\\"
                quoted = c != '"'
            else:
                quoted = c == '"'
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.start():i]


WRITES_M0 = re.compile(r"\bs_\w+\s+m0\s*,")


def test_the_scan_finds_statements():
    text = 'asm volatile("s_mov_b32 m0, %0\\n\\tx (" :: "s"(f(1)) : "memory"); asm("s_nop 0");'
    assert [bool(WRITES_M0.search(s)) for s in statements(text)] == [True, False]


@pytest.mark.parametrize("name", sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*"))))
def test_m0_is_named(name):
    with open(os.path.join(CSRC, name)) as f:
        for s in statements(f.read()):
            if WRITES_M0.search(s):
                assert '"m0"' in s.rsplit(":", 1)[1], s
