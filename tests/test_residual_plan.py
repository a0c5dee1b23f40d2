"""The plan of a GEMM with a residual can be asked for, and a tuning without a choice is none."""
import pytest
import torch

import fp8_block_scaled_bsgemm_b200 as bsg

SIZES = [(8192, 4096, 14336), (2048, 4096, 8192), (2048, 4096, 32768), (1536, 4096, 8192), (1, 7168, 7168), (300, 784, 1040)]


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_plans(gran, M, N, K):
    plain = bsg.make_plan(M, N, K, gran)
    with_residual = bsg.make_plan(M, N, K, gran, residual=True)
    assert bsg.make_plan(M, N, K, gran, residual=True, tuning={}) == with_residual
    if gran != 128:
        assert with_residual == plain
    for tuning in ({"stream_k": -1}, {"variant": "data_parallel"}):
        assert bsg.make_plan(M, N, K, gran, tuning=tuning, residual=True) == bsg.make_plan(M, N, K, gran, tuning=tuning)


def test_where_they_differ():
    assert bsg.make_plan(8192, 4096, 14336)["sk_ctas"] > 0
    assert bsg.make_plan(8192, 4096, 14336, residual=True)["sk_ctas"] == 0
    assert bsg.make_plan(2048, 4096, 32768)["cta_pair"] == 1
    assert bsg.make_plan(2048, 4096, 32768, residual=True)["cta_pair"] == 0
    assert bsg.make_plan(1536, 4096, 8192, residual=True) == bsg.make_plan(1536, 4096, 8192)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(2048, 4096, 8192), (2048, 4096, 32768), (300, 784, 1040)])
def test_a_call_takes_its_plan(M, N, K):
    """FP32 sums in another order differ in their last places somewhere: equal bits say that the plan is the same."""
    gen = torch.Generator(device="cuda").manual_seed(M)
    a, sa = bsg.quantize(torch.randn(M, K, generator=gen, device="cuda"))
    b, sb = bsg.quantize(torch.randn(N, K, generator=gen, device="cuda"))
    residual = torch.randn(M, N, generator=gen, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    kw = dict(out_dtype=torch.float32, residual=residual)
    out = bsg.gemm(a, b, sa, sb, **kw)
    assert torch.equal(out, bsg.gemm(a, b, sa, sb, tuning={}, **kw))
    pl = bsg.make_plan(M, N, K, num_sms=sms, residual=True)
    same = {"variant": "cta_pair" if pl["cta_pair"] else "swap_ab" if pl["swap_ab"] else "data_parallel", "bnq": pl["bnq"],
            "stream_k": 1 if pl["sk_ctas"] else -1}
    if pl["splits"] > 1:
        same = {**same, "splits": pl["splits"], "stream_k": 0}
    assert bsg.make_plan(M, N, K, num_sms=sms, tuning=same) == pl
    assert torch.equal(out, bsg.gemm(a, b, sa, sb, tuning=same, **kw))
