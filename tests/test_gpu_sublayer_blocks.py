"""Matrices with several blocks to a CTA, and rows that a warp takes alone: every element of every row.

The block kernel's CTAs (592 of one block each at g = 64, 296 at g = 128, about 70 clusters at g = 256) walk 2145, 561
and 153 blocks here, so the walk, the fetches ahead and the reuse of every exchanged value are all under way; at 4900
rows the norm's row kernel gives a row to a warp.
"""
import pytest
import torch

import fp8_block_scaled_bsgemm_b200 as bsg

import sublayer_util as su

pytestmark = pytest.mark.gpu

EPS = 1e-6
U = su.U


def gen_of(*seed):
    return torch.Generator(device="cuda").manual_seed(hash(seed) % (1 << 31))


def randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def blocks_of(rows, cols, g):
    return -(-rows // g) * -(-cols // g)


def rstd_bound(cols):
    """Relative bound of rstd for many rows. A thread adds 4 squares of a run, by fused steps, into each half of its
    sum, over its share of the row's runs: the longest chain is a warp's to a row, ceil(cols / 256) runs. One addition
    of the halves, 5 exchanges, up to 8 warps; half of that for the root, then the mean, eps and the root's rounding,
    2 + 2 halves and one."""
    return (4 * -(-cols // 256) + 1 + 5 + 8 + 2) / 2 * U + 2 * U


def check_norm(x, w, r, g, fmt, result):
    q, s, h, rstd = result
    want_h = su.stream(x, r)
    assert torch.equal(h, want_h)
    want = su.norm(want_h, w, EPS)[1]
    assert ((rstd.double() - want).abs() <= rstd_bound(x.shape[1]) * want).all()
    # the kernel's own values, bit for bit, through the quantiser
    want_q, want_s = bsg.quantize((h.float() * rstd[:, None]) * w.float(), g, fmt)
    assert torch.equal(s, want_s)
    bad = q != want_q
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


SIZES = [(2100, 4112), (4900, 400)]
TYPES = [(torch.bfloat16, "e4m3"), (torch.float32, "e5m2")]


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("with_residual", [False, True])
def test_norm(gran, rows, cols, dtype, fmt, with_residual):
    assert rows < 4800 or rows * 32 >= 148 * 1024
    assert rows >= 4800 or blocks_of(rows, cols, gran) > {64: 592, 128: 296, 256: 74}[gran]
    gen = gen_of(gran, rows)
    x = randn(gen, rows, cols, dtype=dtype) * torch.exp2(randn(gen, rows, 1)).to(dtype)
    r = randn(gen, rows, cols, dtype=dtype) if with_residual else None
    w = (1 + 0.3 * randn(gen, cols)).to(dtype)
    check_norm(x, w, r, gran, fmt, bsg.rms_norm_quantize(x, w, residual=r, eps=EPS, gran=gran, fmt=fmt, return_rstd=True))


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("act", ["relu", "gelu"])
def test_activation(gran, dtype, fmt, act):
    rows, cols = SIZES[0]
    gen = gen_of(gran, 2)
    z = randn(gen, rows, cols, dtype=dtype) * torch.exp2(randn(gen, rows, 1)).to(dtype)
    q, s = bsg.activation_quantize(z, act, gran=gran, fmt=fmt)
    if act == "relu":
        want = bsg.quantize(z.clamp(min=0), gran, fmt)
        assert torch.equal(s, want[1]) and torch.equal(q, want[0])
    su.check_codes(q, s, su.act(z, act), gran, fmt, 2 * U, su.gelu_abs(z) if act == "gelu" else None)


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("act", [None, "relu", "gelu"])
def test_activation_backward(gran, dtype, fmt, act):
    rows, cols = SIZES[0]
    gen = gen_of(gran, 3)
    dout = randn(gen, rows, cols, dtype=dtype, scale=0.01)
    z = randn(gen, rows, cols, dtype=dtype, scale=2.0) if act else None
    q, s, db = bsg.activation_backward_quantize(dout, z, act, gran=gran, fmt=fmt)
    dz = dout.double() * su.act_slope(z, act)
    if act != "gelu":
        # (where ReLU's slope is 0 the kernel's value is +0; a product with dout would have dout's sign)
        want = bsg.quantize(dout if act is None else torch.where(z > 0, dout, torch.zeros_like(dout)), gran, fmt)
        assert torch.equal(s, want[1]) and torch.equal(q, want[0])
    extra = dout.double().abs() * su.gelu_slope_abs(z) if act == "gelu" else None
    su.check_codes(q, s, dz, gran, fmt, 3 * U, extra)
    # a column's longest chain: a thread's rows of a block (at most 8), its block's groups of threads (at most 32),
    # then the partial rows: up to 33 row blocks of 4 parts, a 32nd of them at a time, and 32 such sums
    tol = dz.abs().sum(0) * (8 + 32 + 5 + 32) * U + (0 if extra is None else extra.sum(0)) + 2.0 ** -140
    assert ((db.double() - dz.sum(0)).abs() <= tol).all(), float(((db.double() - dz.sum(0)).abs() / tol).max())


@pytest.mark.parametrize("what", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("op", ["relu", "gelu", "backward relu", "backward gelu", "backward none"])
def test_a_value_that_is_not_finite_spoils_its_block_alone(gran, what, op):
    rows, cols = 600, 1040
    gen = gen_of(gran, 4)
    x, z = randn(gen, rows, cols), randn(gen, rows, cols)

    def run(x):
        if op.startswith("backward"):
            act = op.split()[1]
            return bsg.activation_backward_quantize(x, None if act == "none" else z, act, gran=gran)
        return bsg.activation_quantize(x, op, gran=gran)

    clean = run(x)
    bad = x.clone()
    bad[300, 517] = float(what)
    got = run(bad)
    rb, cb = 300 // gran, 517 // gran
    block = torch.zeros(rows, cols, dtype=torch.bool, device="cuda")
    block[rb * gran:(rb + 1) * gran, cb * gran:(cb + 1) * gran] = True
    assert torch.equal(got[0][~block], clean[0][~block])
    s, t = got[1].view(-(-rows // gran), -1).clone(), clean[1].view(-(-rows // gran), -1).clone()
    s[rb, cb] = t[rb, cb] = 0
    assert torch.equal(s, t)
    if len(got) > 2:
        keep = torch.arange(cols, device="cuda") != 517
        assert torch.equal(got[2][keep], clean[2][keep])
