"""Streams given to the operators around the GEMM: torch's, other objects with a handle, and bare handles."""
import pytest
import torch

import fp8_block_scaled_bsgemm_b200 as bsg

pytestmark = pytest.mark.gpu


class OnlyAHandle:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_objects_and_handles():
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(96, 528, generator=gen, device="cuda")
    w = torch.ones(528, device="cuda")
    a, sa = bsg.quantize(x)
    rstd = torch.ones(96, device="cuda")
    b, sb = bsg.quantize(torch.randn(272, 528, generator=gen, device="cuda"))

    def run(stream=None):
        return [*bsg.rms_norm_quantize(x, w, residual=x, return_rstd=True, stream=stream),
                *bsg.rms_norm_backward(x, x, w, rstd, stream=stream),
                bsg.gemm(a, b, sa, sb, stream=stream), *bsg.activation_quantize(x, "relu", stream=stream),
                *bsg.activation_backward_quantize(x, x, "relu", stream=stream)]

    want = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    default = torch.cuda.default_stream()
    # 0, 1 and 2 are CUDA's own names: the default stream, the same, and the calling thread's
    for given in (s, OnlyAHandle(s.cuda_stream), s.cuda_stream, default, OnlyAHandle(0), 0, 1, 2):
        got = run(given)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want)), given
        assert torch.cuda.current_stream() == default
