"""What the compiler is told of the block operators' inline assembly (CPU only; reads the sources)."""
import glob
import os
import re

from sequence_scan_amd import build as lib_build


def asm_statements():
    for path in sorted(glob.glob(os.path.join(lib_build.CSRC, "*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s*(?:volatile\s*)?\(", text):
            depth, i, quoted = 1, m.end(), False
            while depth:
                c = text[i]
                if c == '"':
                    quoted = not quoted
                elif not quoted:
                    depth += (c == "(") - (c == ")")
                i += 1
            yield os.path.basename(path), text[m.start():i]


def test_assembly_that_writes_m0_says_so():
    """m0 is a register of the compiler's too: a statement that writes it has to name it as clobbered."""
    found = [(f, s) for f, s in asm_statements() if re.search(r"\bs_\w+\s+m0,", s)]
    assert found
    for f, s in found:
        assert re.search(r':[^:]*"m0"[^:]*\)$', s), f"{f}: {s}"
