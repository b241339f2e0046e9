"""Inline PTX: every operand that a statement takes stands in its text.  One that does not is computed for nobody: the
assembler sees no use of it and drops what leads to it, an order between instructions that it was to hold included."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "eagle_tree_speculative_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def _statements(text):
    """(line, template, operands) of every asm statement: operands are outputs and inputs in order."""
    text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), text)
    for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
        at, depth, quoted, start = m.end(), 1, False, m.end()
        parts = []                                         # between colons outside strings and brackets
        while depth:
            c = text[at]
            if quoted:
                if c == "\\":
                    at += 1
                quoted = c != '"'
            elif c == '"':
                quoted = True
            elif c in "([{":
                depth += 1
            elif c in ")]}":
                depth -= 1
            elif c == ":" and depth == 1:
                parts.append(text[start:at])
                start = at + 1
            at += 1
        parts.append(text[start:at - 1])
        template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', parts[0]))
        constraints = [c for p in parts[1:3] for c in re.findall(r'"([^"]*)"\s*\(', p)]
        yield text.count("\n", 0, m.start()) + 1, template, constraints


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_every_operand_is_used(path):
    unused = []
    for line, template, constraints in _statements(open(path).read()):
        if not template:                                   # no instruction: hides from the compiler where a value comes from
            continue
        named = {int(x) for x in re.findall(r"(?<!%)%(\d+)", template)}
        assert all(x < len(constraints) for x in named), (line, template)
        unused += [(line, i, c) for i, c in enumerate(constraints) if i not in named]
    assert not unused, f"(line, operand, constraint) {unused}"


def test_the_statements_are_found():
    got = list(_statements('asm volatile(\n "{\\n a %0, [%1];" // x\n " b %%clock;}" ::"r"(f(x, y)), "l"(p), "n"(3) : "memory");'))
    assert [(t[0], len(t[2])) for t in got] == [(1, 3)] and "%0" in got[0][1] and "%%clock" in got[0][1]
    assert sum(len(list(_statements(open(f).read()))) for f in FILES) > 50
