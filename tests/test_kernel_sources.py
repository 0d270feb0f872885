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


def test_inline_assembly_leaves_m0_to_the_compiler():
    """m0 is the compiler's to use: a block that needs it takes it as an operand, and none writes
    it."""
    blocks = list(asm_blocks())
    assert not [b for b in blocks if re.search(r"\bm0,", b[1])]
    fetches = [b for b in blocks if "global_load_lds" in b[1]]
    assert fetches and all('"{m0}"(' in b[1] for b in fetches)
