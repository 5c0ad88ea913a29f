"""The copies into LDS written as inline assembly keep their own wait states (no GPU needed): the compiler inserts none
inside an assembly block and does not see what stands in it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_block_scaled_tensor_amd", "csrc")
# A vector memory instruction reads a scalar register that a vector instruction wrote (v_readlane of a spilled address,
# v_readfirstlane of a uniform one) no sooner than five wait states later.
VALU_SGPR_TO_VMEM = 5


def blocks():
    """(file, instructions) of every assembly block that loads or stores."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        text = open(path, encoding="utf-8").read()
        for m in re.finditer(r"asm(?:\s+volatile)?\s*\(((?:\s*\"[^\"]*\")+)", text):
            code = "".join(re.findall(r'"([^"]*)"', m.group(1))).replace("\\t", " ")
            ins = [i.strip() for i in code.split("\\n") if i.strip()]
            if any(re.match(r"(global|buffer|flat)_", i) for i in ins):
                yield os.path.basename(path), ins


@pytest.mark.parametrize("file,ins", list(blocks()), ids=lambda v: v if isinstance(v, str) else v[-1].split()[0])
def test_a_copy_waits_for_its_address(file, ins):
    at = next(i for i, s in enumerate(ins) if re.match(r"(global|buffer|flat)_", s))
    waits = sum(int(s.split()[1]) + 1 if s.startswith("s_nop") else 1 for s in ins[:at])
    assert waits >= VALU_SGPR_TO_VMEM, (file, ins)


def test_there_are_copies():
    assert len(list(blocks())) == 6
