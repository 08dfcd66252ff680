"""Kernels that allocate TMEM let the next kernel's CTAs come only afterwards. (One of those could take an
SM's columns and then wait, for the kernel before it to end, while a CTA of that kernel waits for columns;
the order is checked in the source because such a hang is not for a GPU to show.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "rmsnorm_precision_activation_gb300", "csrc")


@pytest.mark.parametrize("name", ["rmsq_matmul_tc.cuh", "rmsq_matmul_pair.cuh"])
def test_tmem_is_allocated_before_dependents_may_come(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*", "", text)
    kernel = text[text.index("__global__"):]
    alloc = kernel.index("tcgen05.alloc")
    assert "pdl_wait()" not in kernel[:alloc] and "launch_dependents" not in kernel[:alloc]
    # and every thread gets to the barrier behind the allocation first
    after = kernel[alloc:]
    assert after.index("__syncthreads()") < after.index("pdl_wait()")
