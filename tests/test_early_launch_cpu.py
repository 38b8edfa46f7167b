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


@pytest.mark.parametrize("name", ["common.cuh", "checkpoint.cuh", "norm.cuh", "embedding.cuh", "gemm_sr.cuh"])
def test_no_read_only_loads_in_the_sums_that_start_early(name):
    """The norm's and the embedding's sums start while the kernel ahead writes what they add up, and the bf16 product may
    start while its operands are written; the checkpoint's functions are what the sums load and store with."""
    test_no_read_only_loads_beside_early_launches(name)


def test_every_file_with_early_launches_is_looked_at():
    """All but the 8-bit product of few tokens, whose read-only loads are of the weight and its scales, older than the
    kernel that it may overlap."""
    looked_at = {"product.cuh", "int8_product.cuh", "muon.cuh", "skinny.cuh", "int8.cuh", "norm.cuh", "embedding.cuh", "gemm_sr.cuh"}
    early = set()
    for name in os.listdir(CSRC):
        with open(os.path.join(CSRC, name)) as f:
            if re.search(r"griddepcontrol|launch_early\(", f.read()):
                early.add(name)
    assert early - {"int8_few.cuh"} <= looked_at
