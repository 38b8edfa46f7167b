"""What the sources must hold for kernels that start before the one ahead of
them on the stream has ended."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "stochastic_rounding_gb300", "csrc")


@pytest.mark.parametrize("name", ["product.cuh", "int8_product.cuh", "muon.cuh", "skinny.cuh", "int8.cuh"])
def test_no_read_only_loads_beside_early_launches(name):
    """The read-only path (ld.global.nc, __ldg) is for memory that nobody writes
    while the kernel runs, and is not ordered by griddepcontrol.wait.  The
    products, the scaled copies and the quantisers start while the kernel ahead of
    them writes what they read, so their sources use ordinary loads throughout."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg\s*\(|\bld\.global(\.\w+)*\.nc\b|__restrict__", code)
