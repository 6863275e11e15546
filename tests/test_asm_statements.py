"""What the sources' inline assembly does to registers that the compiler also uses has to be told to it (no GPU here)."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "cnn_convolution_fwd_amd", "csrc")


def statements():
    """(file, text of the instructions, the operand lists after it) of every asm statement."""
    for name in sorted(os.listdir(SRC)):
        with open(os.path.join(SRC, name)) as f:
            source = f.read()
        for m in re.finditer(r"\basm\s+volatile\s*\(", source):
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(source[end], 0)
                end += 1
            body = source[m.end():end - 1]
            first = re.match(r'\s*("(?:[^"\\]|\\.)*"\s*)+', body)
            yield name, re.sub(r"\\[nt]", " ", first.group(0)), body[first.end():]


ALL = list(statements())


def test_there_are_some():
    assert any("lds" in text for _, text, _ in ALL) and any("s_barrier" in text for _, text, _ in ALL)


@pytest.mark.parametrize("name,text,operands", ALL, ids=["%s-%d" % (s[0], i) for i, s in enumerate(ALL)])
def test_m0_is_the_compilers(name, text, operands):
    """No instruction writes m0 behind the compiler's back; a copy to LDS, which reads it, takes it as an operand."""
    assert not re.search(r"\b[sv]_\w+\s+m0\b", text), "%s writes m0" % name
    if re.search(r"\boffen lds\b|\blds\b", text):
        assert '"{m0}"' in operands
    assert "memory" in operands or not re.search(r"\b(buffer|global|ds|flat)_|s_waitcnt|s_barrier", text)
