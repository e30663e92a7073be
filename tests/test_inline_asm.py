"""Inline assembly of the kernels (no GPU): what a statement writes, it says."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "differentiable_gaussian_splat_amd",
                    "csrc")


def statements(path):
    """The asm statements of a source file, from "asm" to the closing semicolon."""
    with open(path) as f:
        return re.findall(r"\basm\b[^;]*?\((?:[^;\"]|\"(?:[^\"\\\\]|\\\\.)*\")*\);", f.read())


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.h*"))), ids=os.path.basename)
def test_written_m0_is_a_clobber(path):
    """A value that the compiler keeps in m0 does not survive a statement that writes it."""
    for s in statements(path):
        if re.search(r"\bs_\w+\s+m0\s*,", s):
            assert re.search(r'"m0"\s*[,)]', s), s


def test_statements_are_found():
    found = statements(os.path.join(CSRC, "labelloss.hip"))
    assert sum("m0," in s for s in found) == 1 and len(found) >= 4
