"""Inline assembly of the kernels says what it writes."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "differentiable_gaussian_splatting_dgs_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip")))


def statements(text):
    """The operands of every asm statement, strings and all, up to its closing parenthesis."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, i, quoted = 1, m.end(), False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.end():i - 1]


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_registers_written_by_name_are_clobbered(path):
    """m0, vcc and exec as destinations, which no operand stands for."""
    with open(path) as f:
        text = f.read()
    for s in statements(text):
        code = s.split(":")[0]
        clobbers = re.findall(r'"([^"]*)"', s.rsplit(":", 1)[1]) if ":" in s else []
        for register in re.findall(r"\b[sv]_\w+\s+(m0|vcc|exec)\s*,", code):
            assert register in clobbers, s
