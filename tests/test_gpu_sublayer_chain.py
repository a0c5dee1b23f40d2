"""Norm -> GEMM and activation -> GEMM on buffers that stay the same while their contents change.

The GEMM is launched beside the kernel that writes its operand and scales; replayed graphs and calls without a
synchronisation between them have to give, bit for bit, what the same calls give one at a time.
"""
import pytest
import torch

import fp8_block_scaled_bsgemm_b200 as bsg

pytestmark = pytest.mark.gpu


def randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("rows,H,F,tuning", [(1, 1040, 2064, None), (40, 1040, 784, None), (300, 784, 1552, None),
                                             (520, 2064, 528, {"variant": "cta_pair"})])
def test_replayed_chain(gran, rows, H, F, tuning):
    gen = torch.Generator(device="cuda").manual_seed(gran + rows)
    bf = torch.bfloat16
    x, r = randn(gen, rows, H, dtype=bf), randn(gen, rows, H, dtype=bf)
    w = randn(gen, H)
    bias = randn(gen, F)
    q1, s1 = bsg.quantize(randn(gen, F, H, scale=0.05), gran)
    q2, s2 = bsg.quantize(randn(gen, H, F, scale=0.05), gran)
    group_m = torch.tensor([rows], dtype=torch.int32, device="cuda")
    rb, kb = -(-rows // gran), -(-H // gran)
    scales = torch.ones((rb + 1) * kb, device="cuda")   # the grouped call's buffer is a row of blocks longer

    def run(between=lambda: None):
        qa, sa, h, _ = bsg.rms_norm_quantize(x, w, residual=r, gran=gran, scales=scales[:rb * kb], return_rstd=True)
        between()
        z = bsg.gemm(qa, q1, sa, s1, gran=gran, bias=bias, tuning=tuning)
        between()
        g = bsg.grouped_gemm(qa, q1[None], scales, s1[None], group_m, gran=gran)
        between()
        qh, sh = bsg.activation_quantize(z, "gelu", gran=gran)
        between()
        out = bsg.gemm(qh, q2, sh, s2, gran=gran, residual=h, tuning=tuning)
        between()
        qd, sd, db = bsg.activation_backward_quantize(out, None, gran=gran)
        between()
        return [qa, sa, h, z, g, qh, sh, out, qd, sd, db]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run()                              # workspaces exist before the capture
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            outs = run()
    torch.cuda.synchronize()
    inputs = [(randn(gen, rows, H, dtype=bf, scale=2.0 ** (k - 4)), randn(gen, rows, H, dtype=bf, scale=2.0 ** (4 - k))) for k in range(8)]
    got = []
    with torch.cuda.stream(side):
        for a, b in inputs:                # no synchronisation between the replays
            x.copy_(a)
            r.copy_(b)
            graph.replay()
            got.append([o.clone() for o in outs])
    torch.cuda.synchronize()
    for (a, b), of in zip(inputs, got):
        x.copy_(a)
        r.copy_(b)
        want = run(torch.cuda.synchronize)
        torch.cuda.synchronize()
        for i, (u, v) in enumerate(zip(of, want)):
            assert torch.equal(u, v), i
    assert bsg.get_last_device_status() == 0
