"""What the kernels' sources have to keep to, read on the CPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kronecker_factored_gptq_amd", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.h*")))


def statements(text):
    """The inside of every asm(...) statement, parentheses balanced."""
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield text[m.end():at - 1]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_inline_assembly_names_the_fixed_registers_it_writes(path):
    """m0, exec and vcc have no operand of their own in most instructions: where a statement's text
    writes one, the compiler has to be told, or it may keep a value of its own there."""
    for s in statements(open(path).read()):
        text = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', s.split("::")[0])).replace("\\n", "\n").replace("\\t", " ")
        for line in text.splitlines():
            written = re.match(r"\s*[sv]_\w+\s+(m0|exec|vcc)\b", line)
            assert not written or '"%s"' % written.group(1) in s, (os.path.basename(path), line)
