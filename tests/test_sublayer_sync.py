"""What a kernel may do before another's memory is in place, read off the sources (no GPU).

A kernel launched with programmatic dependent launch lives beside the one in front of it; a read-only (non-coherent)
load is allowed only for memory that nothing writes during the kernel's life.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scaled_bsgemm_b200", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


# every source whose kernels wait by griddepcontrol.wait
PROGRAMMATIC = ["bsgemm_kernel.cuh", "bsgemm_pair.cuh", "bsgemm_blocks.cuh", "bsgemm_norm.cu", "bsgemm_act.cu", "bsgemm_rows.cuh"]


def test_no_read_only_loads_beside_a_running_writer():
    for name in PROGRAMMATIC:
        text = source(name)
        assert not re.search(r"__ldg\s*\(|ld\.global\.nc|ldu\.global|__restrict__", text), name
    # the other launches have no programmatic attribute, and begin after everything before them
    assert "ProgrammaticStreamSerialization" not in source("bsgemm_quant.cu") + source("bsgemm_noalloc.cu")
