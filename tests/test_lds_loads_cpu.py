"""Loads from memory straight to LDS take their LDS address from m0.  On gfx9 a scalar write of m0 needs one wait state
before such a load; the compiler puts it there between its own instructions, but not inside an inline block."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rotation_bit_ptq_amd", "csrc")
SOURCES = sorted(p for e in ("*.hip", "*.h") for p in glob.glob(os.path.join(CSRC, e)))


def blocks(path):
    """The instructions of a file's inline blocks that write m0."""
    with open(path) as f:
        text = f.read()
    for m in re.finditer(r'asm\s+volatile\s*\(((?:\s*"(?:[^"\\]|\\.)*")+)', text):
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m[1]))
        lines = [x.strip() for x in re.split(r"\\n|\\t", code) if x.strip()]
        if any(re.match(r"s_\w+\s+m0\b", x) for x in lines):
            yield lines


def test_the_scan_finds_the_blocks():
    assert sum(1 for p in SOURCES for _ in blocks(p)) >= 7


@pytest.mark.parametrize("path", [p for p in SOURCES if any(True for _ in blocks(p))], ids=os.path.basename)
def test_a_wait_state_stands_between_m0_and_the_load(path):
    for lines in blocks(path):
        at = next(i for i, x in enumerate(lines) if re.match(r"s_\w+\s+m0\b", x))
        assert lines[at + 1].startswith("s_nop"), lines
