"""GELU in the GEMM's epilogue is one function, whatever the plan and whether a residual is given."""
import pytest
import torch

import fp8_block_scaled_bsgemm_b200 as bsg

import sublayer_util as su

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("tuning,M,N,K", [
    ({"variant": "data_parallel", "bnq": 256, "stream_k": -1}, 300, 784, 1040),
    ({"variant": "data_parallel", "bnq": 128, "splits": 3}, 200, 400, 2064),
    ({"variant": "data_parallel", "bnq": 128, "stream_k": 1}, 640, 784, 1280),
    ({"variant": "swap_ab", "bnq": 32, "stream_k": 1}, 20, 1552, 2064),
    ({"variant": "cta_pair"}, 528, 784, 1280),
])
@pytest.mark.parametrize("with_bias", [False, True])
def test_gelu_beside_a_zero_residual(gran, tuning, M, N, K, with_bias):
    """Adding a residual of zeros changes no bit of an FP32 output (the sign of a zero aside)."""
    gen = torch.Generator(device="cuda").manual_seed(gran + M)
    a, sa = bsg.quantize(torch.randn(M, K, generator=gen, device="cuda"), gran)
    b, sb = bsg.quantize(torch.randn(N, K, generator=gen, device="cuda") * 3 / K ** 0.5, gran)
    bias = torch.randn(N, generator=gen, device="cuda") if with_bias else None
    kw = dict(gran=gran, tuning=tuning, bias=bias, activation="gelu")
    plain = bsg.gemm(a, b, sa, sb, out_dtype=torch.float32, **kw)
    zeros = torch.zeros(M, N, device="cuda")
    got = bsg.gemm(a, b, sa, sb, out_dtype=torch.float32, residual=zeros, **kw)
    bad = got != plain
    assert not bad.any(), (int(bad.sum()), float((got - plain).abs().max()))
    # and it is 1 + erf's: the same products without an activation, in FP32, through the 64-bit form
    z = bsg.gemm(a, b, sa, sb, gran=gran, tuning=tuning, bias=bias, out_dtype=torch.float32)
    # erff is within 2 units of its last place (below 1: 2 U), the sum and the two products one U each of 0.5 (1 + erf)
    assert ((got.double() - su.act(z, "gelu")).abs() <= z.abs().double() * (0.5 * 2 + 3) * su.U).all()
