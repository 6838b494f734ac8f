"""The wait-state check of tests/test_asm_hazards.py for the adapter projection's
tiles, which run the same inline-assembly K loop.  CPU only."""
import os
import tempfile

import pytest

from tests.test_asm_hazards import HIPCC, _compile, _instructions, _violations


@pytest.mark.skipif(HIPCC is None, reason="hipcc not available")
def test_no_valu_write_of_the_tiles_mfma_operands():
    with tempfile.TemporaryDirectory() as d:
        asm = _compile("lora_rows.hip", os.path.join(d, "lora_rows.s"))
    ins, in_asm = _instructions(asm)
    n, bad = _violations(ins, only=in_asm)
    assert not bad, bad[:3]
    assert n > 1000  # the inline-assembly loops were found
