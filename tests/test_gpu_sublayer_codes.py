"""The codes and scales of the norm and activation operators are the quantiser's, bit for bit.

Where a kernel's value is known exactly in FP32 (a gradient passed straight through, a ReLU, a product in a known
order) ``bsg.quantize`` of those values has to give the same bytes: one scale RN(amax / FMAX) and the code of the
correctly rounded quotient.
"""
import pytest
import torch

import fp8_block_scaled_bsgemm_b200 as bsg

import sublayer_util as su

pytestmark = pytest.mark.gpu

EPS = 1e-6


def gen_of(*seed):
    return torch.Generator(device="cuda").manual_seed(hash(seed) % (1 << 31))


def beside_borders(gen, rows, cols, g, fmt, exponent=0):
    """FP32 values of which most lie within two of FP32's steps of a border between two codes."""
    v = torch.rand(rows, cols, generator=gen, device="cuda") + 1.0       # sets each block's amax, in [1, 2)
    amax = su.block_amax(v, g)
    s = (amax.cpu() / su.FMAX[fmt]).cuda()          # divided on the CPU: correctly rounded
    m = su.MANTISSA[fmt]
    e = torch.randint(su.MIN_EXP[fmt], 8 if fmt == "e4m3" else 15, (rows, cols), generator=gen, device="cuda")
    k = torch.randint(0, 1 << m, (rows, cols), generator=gen, device="cuda")
    border = torch.ldexp(1.0 + (2 * k + 1).double() / (2 << m), e)       # half way between neighbours
    near = (border * su.spread(s.double(), g, rows, cols)).float()
    near = (near.view(torch.int32) + torch.randint(-2, 3, (rows, cols), generator=gen, device="cuda", dtype=torch.int32)).view(torch.float32)
    first = torch.zeros(rows, cols, dtype=torch.bool, device="cuda")
    t = v == su.spread(amax, g, rows, cols)         # the largest of each block stays
    first |= t | (near.abs() >= su.spread(amax, g, rows, cols))
    out = torch.where(first, v, near)
    sign = torch.where(torch.rand(rows, cols, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    return torch.ldexp(out * sign, torch.tensor(exponent, device="cuda"))


def same(got, want):
    q, s = got[:2]
    assert torch.equal(s, want[1])
    bad = q != want[0]
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


SIZES = [(130, 1296), (300, 528), (1, 16)]


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_straight_through_codes_beside_borders(gran, fmt, rows, cols):
    gen = gen_of(gran, fmt == "e4m3", rows)
    for exponent in (0, -30, -62, 100, 125):
        x = beside_borders(gen, rows, cols, gran, fmt, exponent)
        x[0, 1:3] = torch.tensor([0.0, -0.0], device="cuda")
        same(bsg.activation_backward_quantize(x, None, gran=gran, fmt=fmt), bsg.quantize(x, gran, fmt))
    # past the range of the corrected product: divisions
    same(bsg.activation_backward_quantize(torch.ldexp(x, torch.tensor(-205, device="cuda")), None, gran=gran, fmt=fmt),
         bsg.quantize(torch.ldexp(x, torch.tensor(-205, device="cuda")), gran, fmt))


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_relu_codes_beside_borders(gran, fmt, rows, cols):
    gen = gen_of(gran, fmt == "e5m2", rows)
    x = beside_borders(gen, rows, cols, gran, fmt)
    same(bsg.activation_quantize(x, "relu", gran=gran, fmt=fmt), bsg.quantize(x.clamp(min=0), gran, fmt))
    z = torch.randn(rows, cols, generator=gen, device="cuda")
    same(bsg.activation_backward_quantize(x, z, "relu", gran=gran, fmt=fmt),
         bsg.quantize(torch.where(z > 0, x, torch.zeros_like(x)), gran, fmt))
    b = x.bfloat16()
    same(bsg.activation_quantize(b, "relu", gran=gran, fmt=fmt), bsg.quantize(b.clamp(min=0), gran, fmt))


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(130, 1296), (300, 528), (1, 7168), (8, 14336)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_codes_are_those_of_its_values(gran, fmt, rows, cols, dtype):
    """y = (h * rstd) * weight, each product rounded once: torch's elementwise products give the same bits."""
    gen = gen_of(gran, rows, cols)
    x = torch.randn(rows, cols, generator=gen, device="cuda").to(dtype)
    w = (1 + 0.3 * torch.randn(cols, generator=gen, device="cuda")).to(dtype)
    q, s, h, rstd = bsg.rms_norm_quantize(x, w, residual=x, eps=EPS, gran=gran, fmt=fmt, return_rstd=True)
    y = (h.float() * rstd[:, None]) * w.float()
    same((q, s), bsg.quantize(y, gran, fmt))
