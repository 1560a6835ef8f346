"""Inline PTX: an asm statement whose instructions read an operand after an earlier one
of its instructions has written a result must mark that result early-clobber ("=&"),
or the compiler may give both one register."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "unet_fa_fwd_gb300", "csrc")
FILES = sorted(f for f in glob.glob(os.path.join(CSRC, "*")) if f.endswith((".inc", ".cuh", ".cu", ".h")))


def _statements(text):
    """(line, instructions, output constraints) of each asm statement with string literals alone."""
    for m in re.finditer(r"\basm(?:\s+volatile)?\s*\(", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0) if text[i] != '"' else 0
            if text[i] == '"':
                i = text.index('"', i + 1)
            i += 1
        body = text[m.end():i - 1]
        at = re.match(r'\s*((?:"[^"]*"\s*)+)', body)
        if not at:
            continue
        code = "".join(re.findall(r'"([^"]*)"', at.group(1)))
        outs = body[at.end():].lstrip()
        outs = outs[1:] if outs.startswith(":") and not outs.startswith("::") else ""
        outs = re.split(r":(?![^(]*\))", outs, maxsplit=1)[0]
        yield (text.count("\n", 0, m.start()) + 1, [s.strip() for s in re.split(r"\\n|;", code) if s.strip()],
               re.findall(r'"([=+&a-z]+)"\s*\(', outs))


def _late_reads(instructions, constraints):
    """Results that are written before another instruction reads an input, not marked early-clobber."""
    n = len(constraints)
    written, bad = set(), set()
    for text in instructions:
        if text.startswith("."):
            continue
        ops = [int(k) for k in re.findall(r"%(\d+)", text)]
        if any(k >= n for k in ops):
            bad |= {k for k in written if "&" not in constraints[k] and "+" not in constraints[k]}
        written |= {k for k in ops if k < n}
    return bad


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_results_are_early_clobber(path):
    found = [(line, sorted(_late_reads(code, outs))) for line, code, outs in _statements(open(path).read())]
    assert not [f for f in found if f[1]]


def test_the_check_sees_such_a_statement():
    text = ('asm volatile("ld.a {%0,%1}, [%4];\\n" "ld.a {%2,%3}, [%5];\\n" "wait;\\n" : "=r"(r[0]), "=r"(r[1]), '
            '"=r"(r[2]), "=r"(r[3]) : "r"(t), "r"(t + (16u << 16)) : "memory");')
    (line, code, outs), = _statements(text)
    assert len(code) == 3 and outs == ["=r"] * 4 and _late_reads(code, outs) == {0, 1}
    (line, code, outs), = _statements(text.replace("=r", "=&r"))
    assert _late_reads(code, outs) == set()
