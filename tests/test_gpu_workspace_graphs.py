"""What the GEMM's workspace holds on to once a graph was captured with it."""
import ctypes

import pytest
import torch

import fp8_block_scaled_bsgemm_b200 as bsg

pytestmark = pytest.mark.gpu

USED_MEM_CURRENT = 7   # cudaMemPoolAttrUsedMemCurrent


def pool_bytes():
    """Bytes that are allocated from the device's stream-ordered pool (the library's workspaces are)."""
    torch.cuda.synchronize()
    rt = ctypes.CDLL("libcudart.so.12")
    pool, used = ctypes.c_void_p(), ctypes.c_uint64()
    assert rt.cudaDeviceGetMemPool(ctypes.byref(pool), torch.cuda.current_device()) == 0
    assert rt.cudaMemPoolGetAttribute(pool, USED_MEM_CURRENT, ctypes.byref(used)) == 0
    return used.value


def operands(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    a, sa = bsg.quantize(torch.randn(M, K, generator=gen, device="cuda"))
    b, sb = bsg.quantize(torch.randn(N, K, generator=gen, device="cuda"))
    return a, b, sa, sb


def test_only_a_buffer_that_a_graph_uses_outlives_its_growth():
    tunings = [{"variant": "data_parallel", "bnq": 128, "splits": s} for s in (2, 4, 8, 16)]
    x = operands(128, 2048, 4096)
    need = [bsg.scratch_bytes(bsg.make_plan(128, 2048, 4096, 128, tuning=t)) for t in tunings]
    assert all(b > 1.25 * a for a, b in zip(need, need[1:]))     # each call outgrows the one before
    bsg.release_workspaces()
    s = torch.cuda.Stream()
    base = pool_bytes()
    with torch.cuda.stream(s):
        want = bsg.gemm(*x, tuning=tunings[0])
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = bsg.gemm(*x, tuning=tunings[0])
        held = []
        for t in tunings[1:]:
            bsg.gemm(*x, tuning=t)
            held.append(pool_bytes() - base)
        g.replay()
        s.synchronize()
    assert torch.equal(out, want)
    # the captured call's buffer and the newest one, a quarter larger than asked for; allocations end on 512 bytes,
    # and the counters are far below a step between two sizes
    for used, n in zip(held, need[1:]):
        assert 1.25 * (need[0] + n) <= used < 1.25 * (need[0] + n) + need[0] / 4, (held, need)
    assert bsg.release_workspaces() == 0     # (by cudaFree, which this count of the pool's does not follow)
    del g
