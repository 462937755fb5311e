"""The example program, with its own check: hidden states served through page steps, cache
writes, paged attention and SSD decode steps against a recomputation from scratch in fp64.
The two round the same values to bf16 (or 8 bits) in each layer, some of them to different
neighbours; the bound is the suite's for bf16 inputs with fp32 state."""
import os
import sys

import pytest

from helpers import TOL_BF16, report

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "f8"])
def test_hybrid_decode(cuda_device, cache):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_decode
    worst = hybrid_decode.main(["--check", "--steps", "9", "--cache", cache])
    report("hybrid example " + cache, hidden=worst)
    assert 0.0 < worst <= TOL_BF16
