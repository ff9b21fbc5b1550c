"""Wait states that inline assembly has to bring along itself (the compiler adds
none inside it), checked in the sources."""
from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_int8_quantized_qk_amd", "csrc")


def blocks():
    """(file, instructions) of every asm statement that has any."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for found in re.finditer(r"\basm\s*(?:volatile)?\s*\(((?:\s*\"(?:[^\"\\]|\\.)*\")+)", text):
            code = "".join(re.findall(r"\"((?:[^\"\\]|\\.)*)\"", found.group(1)))
            lines = [x.strip() for x in re.split(r"\\n|\\t|;", code) if x.strip()]
            if lines:
                yield name, lines


def test_blocks_are_found():
    assert any(any("load_lds" in x for x in lines) for _, lines in blocks())


@pytest.mark.parametrize("name,lines", list(blocks()), ids=lambda v: v if isinstance(v, str) else v[0].split()[0])
def test_m0_is_a_wait_state_old_when_a_load_into_lds_reads_it(name, lines):
    for i, line in enumerate(lines):
        if re.search(r"load_lds|\blds\b", line) and "load" in line:
            before = lines[:i]
            writes = [j for j, x in enumerate(before) if re.match(r"s_\w+\s+m0\b", x)]
            assert writes, f"{name}: {line}: m0 comes from elsewhere, which the compiler cannot wait for"
            assert i - writes[-1] > 1, f"{name}: {line} follows {before[writes[-1]]} at once"
