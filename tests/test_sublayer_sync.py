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


def kernels(text):
    """Name -> body of every kernel of a source."""
    parts = re.split(r"__global__", text)[1:]
    return {re.search(r"\b(\w+_kernel)\s*\(", part).group(1): part for part in parts}


def test_clusters_are_open_before_a_store_to_a_peer():
    """A peer's shared memory is written only past a cluster barrier: arrive, then wait, then the first remote store."""
    found = []
    for name in PROGRAMMATIC + ["bsgemm_quant.cu"]:
        for kernel, body in kernels(source(name)).items():
            store = re.search(r"\b(st_cluster_f32|st_shared_cluster_f32|mbar_arrive_cluster)\s*\(", body)
            if store is None:
                continue
            found.append(kernel)
            head = body[:store.start()]
            opened = "cluster_sync_all(" in head
            arrive, wait = head.find("cluster_open_arrive("), head.find("cluster_open_wait(")
            assert opened or 0 <= arrive < wait, kernel
            # the two halves are run by the same threads: under the same condition
            if not opened:
                def condition(at):
                    return re.search(r"if (?:constexpr )?\(([^;{}]*)\)\s*(?:\{[^{}]*)?(?:bsg::)?$", head[:at]).group(1).strip()
                assert condition(arrive) == condition(wait) or condition(wait) in ("kP > 1",), kernel
    assert sorted(found) == ["block_quant_kernel", "bsgemm_pair_kernel", "norm_backward_kernel", "norm_few_kernel", "quant_kernel"]


def test_nothing_is_left_behind_in_l2():
    """No kernel stores or reads data as the last to leave L2: the places would be lost to the kernels that follow."""
    for name in os.listdir(CSRC):
        assert not re.search(r"evict_last|createpolicy|persisting", source(name)), name
