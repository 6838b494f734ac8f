"""The wait-state check of tests/test_asm_hazards.py for the tiles of the 8-bit products and
of the orthogonalisation, which run the same inline-assembly K loop.  CPU only."""
import os
import tempfile

import pytest

from tests.test_asm_hazards import HIPCC, _compile, _instructions, _violations


@pytest.mark.skipif(HIPCC is None, reason="hipcc not available")
@pytest.mark.parametrize("source", ["int8.hip", "orthogonal.hip"])
def test_no_valu_write_of_the_tiles_mfma_operands(source):
    with tempfile.TemporaryDirectory() as d:
        asm = _compile(source, os.path.join(d, "out.s"))
    ins, in_asm = _instructions(asm)
    n, bad = _violations(ins, only=in_asm)
    assert not bad, bad[:3]
    assert n > 500  # the inline-assembly loops were found
