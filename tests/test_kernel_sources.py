"""What the kernels' sources promise the compiler."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "maxsim_scoring_fwd_amd", "csrc")


def asm_blocks():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\b[^(]*\((.*?)\);", text, re.S):
            yield os.path.basename(path), m.group(1)


def test_registers_written_by_inline_assembly_are_declared():
    """m0 is the compiler's to use: a block that writes it lists it among its clobbers."""
    writes = [(f, b) for f, b in asm_blocks() if re.search(r"\bm0,", b)]
    assert writes, "no such block: drop this test"
    for f, block in writes:
        assert block.rstrip().endswith(': "m0"'), f"{f}: {block}"
