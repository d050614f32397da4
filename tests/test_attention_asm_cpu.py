"""Inline assembly of the kernels' sources: what a statement writes beside its
outputs it declares (CPU only, on the text)."""
from __future__ import annotations

import os
import re

from int4_row_wise_amd import build as qbuild


def statements():
    """(file, template, the statement's other parts) of every asm statement."""
    found = []
    for d, _, files in os.walk(qbuild.CSRC):
        for name in sorted(files):
            with open(os.path.join(d, name)) as f:
                src = re.sub(r"//[^\n]*", "", f.read())
            for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\)\s*;", src, re.S):
                template, _, rest = m.group(1).partition(":")
                found.append((name, template, rest))
    return found


def test_statements_that_use_m0_say_so():
    """A load to LDS takes its address from m0: that is the statement's operand,
    and no statement writes m0 behind the compiler's back."""
    loads = [s for s in statements() if re.search(r"\bm0\b|\blds\b", s[1])]
    assert loads, "no statement loads to LDS: this test reads the sources wrongly"
    for name, template, rest in loads:
        assert not re.search(r"\bs_\w+\s+m0\b", template) or '"m0"' in rest.rsplit(":", 1)[-1], (name, template.strip())
        assert '"{m0}"' in rest or '"m0"' in rest.rsplit(":", 1)[-1], (name, template.strip())
