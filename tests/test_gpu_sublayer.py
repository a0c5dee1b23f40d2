"""The operators around the GEMM on a B200, against plain 64-bit forms (tests/sublayer_util.py)."""
import os
import subprocess
import sys

import pytest
import torch

import fp8_block_scaled_bsgemm_b200 as bsg

import sublayer_util as su

pytestmark = pytest.mark.gpu

EPS = 1e-6


def randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def gen_of(*seed):
    return torch.Generator(device="cuda").manual_seed(hash(seed) % (1 << 31))


# ------------------------------------------------------------------ norm


def check_norm(x, w, residual, gran, fmt, result):
    q, s, h, rstd = result
    rows, cols = x.shape
    want_h = su.stream(x, residual)
    assert torch.equal(h, want_h)
    y, want_rstd = su.norm(want_h, w, EPS)
    rel = su.rstd_rel(cols, gran)
    assert ((rstd.double() - want_rstd).abs() <= rel * want_rstd).all()
    su.check_codes(q, s, y, gran, fmt, rel + 2 * su.U)


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("rows,cols", [(1, 16), (70, 1072), (70, 1264), (1, 7168), (2, 1040), (9, 208), (33, 4112), (64, 64), (130, 1296), (300, 528),
                                       (257, 2064), (5, 40016)])
@pytest.mark.parametrize("dtype,with_residual,fmt", [(torch.bfloat16, True, "e4m3"), (torch.bfloat16, False, "e5m2"),
                                                     (torch.float32, True, "e5m2"), (torch.float32, False, "e4m3")])
def test_norm(gran, rows, cols, dtype, with_residual, fmt):
    gen = gen_of(gran, rows, cols, with_residual)
    x = randn(gen, rows, cols, dtype=dtype, scale=3.0)
    r = randn(gen, rows, cols, dtype=dtype) if with_residual else None
    w = 1 + 0.3 * randn(gen, cols)
    result = bsg.rms_norm_quantize(x, w.to(dtype), residual=r, eps=EPS, gran=gran, fmt=fmt, return_rstd=True)
    check_norm(x, w.to(dtype), r, gran, fmt, result)


def test_norm_mixed_weight_types_and_in_place():
    gen = gen_of(1)
    x, r = randn(gen, 70, 528, dtype=torch.bfloat16), randn(gen, 70, 528, dtype=torch.bfloat16)
    w = randn(gen, 528)
    want = bsg.rms_norm_quantize(x, w, residual=r, eps=EPS, return_rstd=True)
    check_norm(x, w, r, 128, "e4m3", want)
    for into in ("x", "residual"):
        x2, r2 = x.clone(), r.clone()
        got = bsg.rms_norm_quantize(x2, w, residual=r2, eps=EPS, return_rstd=True, residual_out=x2 if into == "x" else r2)
        assert got[2] is (x2 if into == "x" else r2)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    xf = randn(gen, 70, 528)
    check_norm(xf, w.bfloat16(), None, 64, "e4m3",
               bsg.rms_norm_quantize(xf, w.bfloat16(), eps=EPS, gran=64, return_rstd=True))


@pytest.mark.parametrize("gran", [64, 128, 256])
def test_norm_zero_rows_tiny_and_large_values(gran):
    gen = gen_of(2, gran)
    x = randn(gen, 300, 272)
    x[: min(gran, 200)] = 0                     # whole blocks of zeros: scale 1, codes 0
    x[210] = 1e-30                              # far below eps
    x[211] *= 2.0 ** 50
    x[212, 5] = 0
    w = randn(gen, 272)
    w[64:128] = 0
    w[130] = 1e-38
    result = bsg.rms_norm_quantize(x, w, eps=EPS, gran=gran, return_rstd=True)
    check_norm(x, w, None, gran, "e4m3", result)
    if gran <= 128:
        assert (result[1][0] == 1).all() and (result[0][:gran] & 0x7F == 0).all()   # -0 where the weight is negative
    # a weight so small that amax / FMAX is below FP32: scale 1, codes 0
    q, s, _ = bsg.rms_norm_quantize(x[212:], torch.full((272,), 1e-44, device="cuda"), eps=EPS, gran=gran)
    assert (s == 1).all() and (q & 0x7F == 0).all()
    # one step of FP32 above it: scales of a few steps, quotients by division
    w = torch.full((272,), 1e-41, device="cuda")
    q, s, h, rstd = bsg.rms_norm_quantize(x[212:], w, eps=EPS, gran=gran, return_rstd=True)
    y = x[212:].double() * rstd.double()[:, None] * w.double()
    assert (s > 0).all() and (s < 1e-40).all()
    got = su.dequantize(q, s, gran, "e4m3")
    # y itself is rounded to FP32's smallest step, and so is the scale: up to a third of it at 3 steps
    amax = su.spread(su.block_amax(y, gran), gran, *y.shape)
    assert ((got - y).abs() <= amax * 0.5 + 2.0 ** -148).all()


def test_norm_non_finite_rows_spoil_no_other_row():
    gen = gen_of(3)
    x = randn(gen, 256, 256)
    clean = bsg.rms_norm_quantize(x, torch.ones(256, device="cuda"), eps=EPS, return_rstd=True)
    bad = x.clone()
    bad[7, 3] = float("nan")
    q, s, h, rstd = bsg.rms_norm_quantize(bad, torch.ones(256, device="cuda"), eps=EPS, return_rstd=True)
    keep = torch.arange(256, device="cuda") != 7
    assert torch.equal(rstd[keep], clean[3][keep]) and torch.isnan(rstd[7])
    assert torch.isfinite(s).all() and torch.isnan(su.dequantize(q, s, 128, "e4m3")[7]).all()
    assert torch.equal(q[128:], clean[0][128:]) and torch.equal(s[1], clean[1][1])


# ------------------------------------------------------------------ norm's gradient


def bwd_depth(rows, cols):
    """Additions in a row: 8 in a run, 5 in the warp, up to 16 warps and 16 CTAs. In a column: a part's
    rows (each an addition), up to 16 row groups, up to 640 parts."""
    return 8 + 5 + 16 + 16, rows + 16 + 640


def check_norm_backward(dy, h, w, rstd, skip, dx, dw):
    rows, cols = dy.shape
    want_dx, want_dw = su.norm_backward(dy, h, w, rstd, skip)
    n = h.double() * rstd.double()[:, None]
    dn = dy.double() * w.double()
    row_depth, col_depth = bwd_depth(rows, cols)
    r = rstd.double()[:, None]
    mean_abs = (dn * n).abs().mean(1, keepdim=True)
    # r (dn - n m): dn one rounding, n two, m its sum's and three more; then the subtraction and the product by r
    tol = r * (dn.abs() * 3 + n.abs() * mean_abs * (row_depth + 8)) * su.U
    if skip is not None:
        tol = tol + (want_dx.abs() + skip.double().abs()) * su.U
    tol = tol + (want_dx.abs() + tol) * su.out_rounding(dy.dtype) + 2.0 ** -140
    assert ((dx.double() - want_dx).abs() <= tol).all(), float(((dx.double() - want_dx).abs() / tol).max())
    terms = (dy.double() * n).abs().sum(0)
    tol = terms * (col_depth + 3) * su.U + 2.0 ** -140
    assert ((dw.double() - want_dw).abs() <= tol).all(), float(((dw.double() - want_dw).abs() / tol).max())


@pytest.mark.parametrize("rows,cols", [(1, 16), (70, 1072), (21, 1264), (1, 7168), (2, 208), (7, 272), (333, 1552), (1200, 4096), (600, 4112), (40, 16400),
                                       (9, 65536), (5000, 64)])
@pytest.mark.parametrize("dtype,with_skip", [(torch.bfloat16, True), (torch.bfloat16, False), (torch.float32, True),
                                             (torch.float32, False)])
def test_norm_backward(rows, cols, dtype, with_skip):
    gen = gen_of(rows, cols, with_skip)
    h = randn(gen, rows, cols, dtype=dtype, scale=2.0)
    dy = randn(gen, rows, cols, dtype=dtype, scale=0.01)
    skip = randn(gen, rows, cols, dtype=dtype, scale=0.01) if with_skip else None
    w = (1 + 0.3 * randn(gen, cols)).to(dtype)
    rstd = su.norm(h, w, EPS)[1].float()
    dx, dw = bsg.rms_norm_backward(dy, h, w, rstd, dresidual=skip)
    assert dx.dtype == dtype and dw.dtype == torch.float32 and dw.shape == (cols,)
    check_norm_backward(dy, h, w, rstd, skip, dx, dw)
    again = bsg.rms_norm_backward(dy, h, w, rstd, dresidual=skip)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("cols", [528, 8208])
def test_norm_backward_in_place(cols):
    gen = gen_of(4, cols)
    h, dy, skip = (randn(gen, 50, cols, dtype=torch.bfloat16) for _ in range(3))
    w = randn(gen, cols)
    rstd = su.norm(h, w, EPS)[1].float()
    want = bsg.rms_norm_backward(dy, h, w, rstd, dresidual=skip)
    check_norm_backward(dy, h, w, rstd, skip, *want)
    for into in (0, 1):
        a, b = dy.clone(), skip.clone()
        dx, dw = bsg.rms_norm_backward(a, h, w, rstd, dresidual=b, dx=(a, b)[into])
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_norm_backward_against_differences():
    """The forward's FP32 rows, moved by hand: dx against central differences of the 64-bit loss at the kernel's h."""
    gen = gen_of(5)
    h = randn(gen, 3, 64)
    w = randn(gen, 64)
    dy = randn(gen, 3, 64)
    rstd = bsg.rms_norm_quantize(h, w, eps=EPS, return_rstd=True)[3]
    dx, dw = bsg.rms_norm_backward(dy, h, w, rstd)
    d = 1e-6
    for i, j in [(0, 0), (1, 31), (2, 63)]:
        e = torch.zeros(3, 64, dtype=torch.float64, device="cuda")
        e[i, j] = d
        num = ((su.norm(h.double() + e, w, EPS)[0] - su.norm(h.double() - e, w, EPS)[0]) * dy.double()).sum() / (2 * d)
        # the gradient's size here is about 1: 100 FP32 roundings, and the difference's own 1e-8
        assert abs(float(num) - float(dx[i, j])) < 1e-5


# ------------------------------------------------------------------ activations


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("rows,cols", [(1, 16), (70, 1072), (70, 1264), (1, 14336), (8, 272), (130, 1040), (300, 528), (257, 64)])
@pytest.mark.parametrize("dtype,act,fmt", [(torch.bfloat16, "gelu", "e4m3"), (torch.bfloat16, "relu", "e5m2"),
                                           (torch.float32, "gelu", "e5m2"), (torch.float32, "relu", "e4m3")])
def test_activation_quantize(gran, rows, cols, dtype, act, fmt):
    gen = gen_of(gran, rows, cols)
    z = randn(gen, rows, cols, dtype=dtype, scale=2.0)
    q, s = bsg.activation_quantize(z, act, gran=gran, fmt=fmt)
    y = su.act(z, act)
    su.check_codes(q, s, y, gran, fmt, 2 * su.U, su.gelu_abs(z) if act == "gelu" else None)


def test_gelu_over_every_bf16_value():
    """Every finite BF16 z, forward and backward (a gradient of 1 beside each), zeros, denormals and the largest included."""
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32)
    z = bits.to(torch.int16).view(torch.bfloat16)
    z = z[torch.isfinite(z)]
    order = torch.argsort(z.float().abs())      # blocks of like magnitudes, so that none is lost beside a large one
    z = z[order]
    z = torch.cat([z, torch.zeros(-len(z) % 4096, device="cuda", dtype=torch.bfloat16)]).view(-1, 64).contiguous()
    q, s = bsg.activation_quantize(z, "gelu", gran=64)
    su.check_codes(q, s, su.act(z, "gelu"), 64, "e4m3", 4 * su.U, su.gelu_abs(z))
    one = torch.ones_like(z)
    q, s, db = bsg.activation_backward_quantize(one, z, "gelu", gran=64)
    slope = su.act_slope(z, "gelu")
    su.check_codes(q, s, slope, 64, "e4m3", 4 * su.U, su.gelu_slope_abs(z))
    assert ((db.double() - slope.sum(0)).abs() <= su.gelu_slope_abs(z).sum(0) + slope.abs().sum(0) * (z.shape[0]) * su.U).all()


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("rows,cols", [(1, 16), (70, 1072), (70, 1264), (3, 14336), (130, 1040), (300, 528), (777, 64)])
@pytest.mark.parametrize("dtype,act,fmt", [(torch.bfloat16, "gelu", "e5m2"), (torch.bfloat16, "relu", "e4m3"),
                                           (torch.float32, "gelu", "e4m3"), (torch.float32, None, "e5m2"),
                                           (torch.bfloat16, "none", "e4m3")])
def test_activation_backward(gran, rows, cols, dtype, act, fmt):
    gen = gen_of(gran, rows, cols, 7)
    z = randn(gen, rows, cols, dtype=dtype, scale=2.0) if act in ("gelu", "relu") else None
    if z is not None:
        z[0, 3] = 0
    dout = randn(gen, rows, cols, dtype=dtype, scale=0.01)
    q, s, db = bsg.activation_backward_quantize(dout, z, act, gran=gran, fmt=fmt)
    dz = dout.double() * su.act_slope(z, act)
    extra = dout.double().abs() * su.gelu_slope_abs(z) if act == "gelu" else None
    su.check_codes(q, s, dz, gran, fmt, 3 * su.U, extra)
    # a column is added over its block's rows, 16 warps and the parts: no chain longer than the rows and 16 + 32
    tol = dz.abs().sum(0) * (min(rows, 256) + 48 + rows / 32) * su.U + (0 if extra is None else extra.sum(0)) + 2.0 ** -140
    assert ((db.double() - dz.sum(0)).abs() <= tol).all(), float(((db.double() - dz.sum(0)).abs() / tol).max())
    q2, s2, none = bsg.activation_backward_quantize(dout, z, act, gran=gran, fmt=fmt, bias_grad=False)
    assert none is None and torch.equal(q, q2) and torch.equal(s, s2)


def test_activation_backward_zero_block():
    z = torch.full((128, 128), -3.0, device="cuda")
    q, s, db = bsg.activation_backward_quantize(torch.ones_like(z), z, "relu")
    assert (q & 0x7F == 0).all() and (s == 1).all() and (db == 0).all()


# ------------------------------------------------------------------ GEMM with a residual


def gemm_inputs(gen, M, N, K, layout, gran, a_fmt="e4m3"):
    a, sa = bsg.quantize(randn(gen, M, K), gran, a_fmt)
    b, sb = bsg.quantize(randn(gen, N, K, scale=0.05), gran)
    A, B = su.dequantize(a, sa, gran, a_fmt), su.dequantize(b, sb, gran, "e4m3")
    if layout[0] == "t":
        a = a.t().contiguous()
    if layout[1] == "n":
        b = b.t().contiguous()
    return a, b, sa, sb, A, B


def check_gemm(out, A, B, bias, act, residual):
    acc = A @ B.t()
    z = acc if bias is None else acc + bias.double()
    want = su.act(z, act) + residual.double()
    # acc: the tensor core adds 32 products at a time, taken as keeping 22 bits, then FP32 additions over the K
    # blocks and up to 148 pieces; |act'| <= 1.13, the activation's own roundings 4 U, bias and residual one each
    K = A.shape[1]
    mag = A.abs() @ B.abs().t()
    tol = 1.13 * (mag * (K / 32 * 2.0 ** -22 + (K / 64 + 148) * su.U) + (z.abs() * 5 * su.U)) + want.abs() * su.U
    tol = tol + (want.abs() + tol) * su.out_rounding(out.dtype)
    err = (out.double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())


PLANS = [
    (None, 1, 528, 1040, "nt"), (None, 7, 2048, 7168, "nn"), (None, 64, 272, 528, "nt"), (None, 16, 144, 2064, "tt"),
    ({"variant": "swap_ab", "bnq": 128}, 100, 144, 1040, "nt"),
    ({"variant": "swap_ab", "bnq": 32, "splits": 3}, 48, 784, 1280, "tn"),
    ({"variant": "swap_ab", "bnq": 64, "stream_k": 1}, 33, 1552, 2064, "nt"),
    (None, 130, 784, 1296, "nt"), (None, 300, 1552, 528, "nn"), (None, 2048, 2064, 272, "nt"),
    ({"variant": "data_parallel", "bnq": 128, "splits": 4}, 200, 144, 2064, "nn"),
    ({"variant": "data_parallel", "bnq": 256, "stream_k": 1}, 640, 1040, 4112, "tt"),
    ({"variant": "data_parallel", "bnq": 128, "stream_k": 1}, 640, 784, 1280, "nn"),
    ({"variant": "cta_pair"}, 528, 784, 1280, "tn"),
]


@pytest.mark.parametrize("gran", [64, 128, 256])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tuning,M,N,K,layout", PLANS)
def test_gemm_residual(gran, out_dtype, tuning, M, N, K, layout):
    gen = gen_of(gran, M, N, K)
    a, b, sa, sb, A, B = gemm_inputs(gen, M, N, K, layout, gran)
    residual = randn(gen, M, N, dtype=out_dtype, scale=4.0)
    bias = randn(gen, N)
    for act, with_bias in ((None, False), ("relu", True), ("gelu", True), (None, True)):
        kw = dict(layout=layout, gran=gran, tuning=tuning, bias=bias if with_bias else None, activation=act, out_dtype=out_dtype)
        out = bsg.gemm(a, b, sa, sb, residual=residual, **kw)
        check_gemm(out, A, B, bias if with_bias else None, act, residual)
        # in place: bit for bit the same
        inout = residual.clone()
        got = bsg.gemm(a, b, sa, sb, residual=inout, out=inout, **kw)
        assert got is inout and torch.equal(inout, out)
    assert bsg.get_last_device_status() == 0


@pytest.mark.parametrize("M,N,K,gran,tuning", [
    (4096, 4096, 4096, 128, None), (2048, 4096, 14336, 128, None), (4096, 4096, 2064, 64, None), (4096, 4096, 4096, 256, None),
    (4096, 4096, 2064, 128, {"variant": "cta_pair"}), (4096, 4096, 4096, 64, {"variant": "data_parallel", "bnq": 256, "stream_k": -1}),
    (4096, 4096, 1040, 128, {"variant": "data_parallel", "bnq": 128, "stream_k": -1}),
    (4096, 4096, 400, 128, None), (4096, 2064, 144, 64, None)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_gemm_residual_on_many_tiles(M, N, K, gran, tuning, out_dtype):
    """Persistent CTAs walk several tiles, each with its residual on its way in the last K-blocks: every element, four
    times over, against the FP32 product without a residual.

    The two sum the same block products; the residual joins some K-blocks before the end, so the additions after it,
    kGap * kChunks <= 12 of them and the bias's, round a sum that holds it: 14 U (|residual| + sum |a b|), and the
    output's own rounding. The plain product's additions may be ordered otherwise (stream-K): K / 64 U sum |a b|.
    """
    gen = gen_of(17, M, K)
    a, b, sa, sb, A, B = gemm_inputs(gen, M, N, K, "nt", gran)
    mag = A.float().abs() @ B.float().abs().t()
    del A, B
    bias = randn(gen, N)
    base = bsg.gemm(a, b, sa, sb, gran=gran, out_dtype=torch.float32).double()
    for k in range(4):
        residual = randn(gen, M, N, dtype=out_dtype, scale=20.0)
        kw = dict(bias=bias) if k & 1 else {}
        out = bsg.gemm(a, b, sa, sb, gran=gran, tuning=tuning, out_dtype=out_dtype, residual=residual, **kw)
        want = base + residual.double() + (bias.double() if kw else 0)
        tol = (14 * (residual.double().abs() + mag) + K / 64 * mag + (bias.abs() if kw else 0)) * su.U
        tol = tol + (want.abs() + tol) * su.out_rounding(out_dtype)
        bad = (out.double() - want).abs() > tol
        assert not bad.any(), (k, int(bad.sum()), bad.nonzero()[:4].tolist())


def test_gemm_residual_leaves_what_lies_behind_the_output():
    gen = gen_of(8)
    a, b, sa, sb, A, B = gemm_inputs(gen, 130, 264, 272, "nt", 128)
    buf = randn(gen, 140, 264, dtype=torch.bfloat16)
    keep = buf.clone()
    bsg.gemm(a, b, sa, sb, residual=buf[:130], out=buf[:130])
    check_gemm(buf[:130], A, B, None, None, keep[:130])
    assert torch.equal(buf[130:], keep[130:])


def test_gemm_residual_refusals_in_the_binding():
    gen = gen_of(9)
    a, b, sa, sb, A, B = gemm_inputs(gen, 16, 64, 64, "nt", 128)
    r = torch.zeros((16, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (r.float(), r[:8], r.t(), r.cpu(), r.view(64, 16)):
        with pytest.raises(ValueError):
            bsg.gemm(a, b, sa, sb, residual=bad)
    flat = torch.zeros(16 * 64 + 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(bsg.BsgemmError):
        bsg.gemm(a, b, sa, sb, residual=flat[:1024].view(16, 64), out=flat[64:1088].view(16, 64))
    out = bsg.gemm(a, b, sa, sb, residual=r)
    assert torch.equal(out, bsg.gemm(a, b, sa, sb))


# ------------------------------------------------------------------ refusals, streams, graphs


def test_refusals_in_the_binding():
    x = torch.zeros((64, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    rstd = torch.ones(64, device="cuda")
    for call in (lambda: bsg.rms_norm_quantize(x.t()[:32], w), lambda: bsg.rms_norm_quantize(x[0], w),
                 lambda: bsg.rms_norm_quantize(x, w[:32]), lambda: bsg.rms_norm_quantize(x, w, residual=x[:32]),
                 lambda: bsg.rms_norm_quantize(x, w, residual_out=x), lambda: bsg.rms_norm_quantize(x, w, fmt="e3m4"),
                 lambda: bsg.rms_norm_quantize(x, w, q=torch.zeros(8, dtype=torch.uint8, device="cuda")),
                 lambda: bsg.rms_norm_backward(x, x[:32], w, rstd), lambda: bsg.rms_norm_backward(x, x, w, rstd[:3]),
                 lambda: bsg.rms_norm_backward(x, x, w, rstd.double()),
                 lambda: bsg.activation_quantize(x, "swish"), lambda: bsg.activation_backward_quantize(x, None, "gelu"),
                 lambda: bsg.activation_backward_quantize(x, x, None),
                 lambda: bsg.activation_backward_quantize(x, x, "gelu", bias_grad=False, dbias=w)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bsg.rms_norm_quantize(x.half(), w), lambda: bsg.rms_norm_quantize(x, w.half()),
                 lambda: bsg.rms_norm_quantize(x, w, residual=x.bfloat16()),
                 lambda: bsg.rms_norm_backward(x, x.bfloat16(), w, rstd)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: bsg.rms_norm_quantize(x, w, gran=32), lambda: bsg.rms_norm_quantize(x, w, eps=0),
                 lambda: bsg.rms_norm_quantize(torch.zeros((0, 64), device="cuda"), w),
                 lambda: bsg.rms_norm_quantize(x[:, :24].contiguous(), w[:24]),
                 lambda: bsg.activation_quantize(x, None), lambda: bsg.activation_quantize(x, "gelu", gran=100),
                 lambda: bsg.rms_norm_backward(x, x, w, rstd, dx=x)):
        with pytest.raises(bsg.BsgemmError):
            call()


def all_calls(gen):
    """One call of each operator on inputs of its own: a function that returns its outputs."""
    x, r, dy = (randn(gen, 300, 4112, dtype=torch.bfloat16) for _ in range(3))
    w = randn(gen, 4112)
    rstd = su.norm(x, w, EPS)[1].float()
    a, b, sa, sb, _, _ = gemm_inputs(gen, 130, 784, 1040, "nt", 128)
    res = randn(gen, 130, 784, dtype=torch.bfloat16)

    def run(stream=None):
        return [*bsg.rms_norm_quantize(x, w, residual=r, return_rstd=True, stream=stream),
                *bsg.rms_norm_backward(dy, x, w, rstd, dresidual=r, stream=stream),
                bsg.gemm(a, b, sa, sb, residual=res, stream=stream),
                *bsg.activation_quantize(x, "gelu", stream=stream),
                *bsg.activation_backward_quantize(dy, x, "gelu", stream=stream)]

    return run


def test_side_streams():
    """A stream given by object and by handle, its calls ordered on it; the caller's stream is not touched."""
    run = all_calls(gen_of(10))
    want = run()
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        for given in (s, s.cuda_stream):
            got = run(given)
            s.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(got, want))
    # interleaved on two streams: no scratch is shared
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    other = all_calls(gen_of(11))
    want2 = other()
    torch.cuda.synchronize()
    pairs = [(run(s1), other(s2)) for _ in range(5)]
    torch.cuda.synchronize()
    for g1, g2 in pairs:
        assert all(torch.equal(u, v) for u, v in zip(g1, want))
        assert all(torch.equal(u, v) for u, v in zip(g2, want2))


def test_graphs():
    """The calls captured, replayed on new inputs, and two graphs replayed at the same time on two streams."""
    gen = gen_of(12)
    graphs, outs, wants, ins = [], [], [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        x, dy = (randn(gen, 700, 2064, dtype=torch.bfloat16) for _ in range(2))
        w = randn(gen, 2064)

        def run(x=x, dy=dy, w=w):
            q, sc, h, rstd = bsg.rms_norm_quantize(x, w, residual=dy, return_rstd=True)
            dx, dw = bsg.rms_norm_backward(dy, h, w, rstd)
            return [q, sc, h, rstd, dx, dw, *bsg.activation_quantize(x, "gelu"), *bsg.activation_backward_quantize(dy, x, "gelu")]

        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(run())
        x.copy_(randn(gen, 700, 2064, dtype=torch.bfloat16))
        wants.append([t.clone() for t in run()])
        graphs.append(g)
        ins.append((x, dy, w))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_both_marshallings_agree(monkeypatch):
    """The C++ marshalling takes the usual calls, and gives what the Python code gives."""
    run = all_calls(gen_of(14))
    assert bsg._marshal() is not None
    want = run()
    monkeypatch.setattr(bsg, "_fast", None)
    got = run()
    assert len(got) == len(want)
    for u, v in zip(got, want):
        assert u.dtype == v.dtype and u.shape == v.shape and torch.equal(u, v)
    gen = gen_of(15)
    a, b, sa, sb, _, _ = gemm_inputs(gen, 48, 272, 144, "tn", 64, "e5m2")
    a = a.view(torch.float8_e5m2)
    bias, res = randn(gen, 272), randn(gen, 48, 272)
    kw = dict(layout="tn", gran=64, bias=bias, activation="gelu", out_dtype=torch.float32, residual=res)
    slow = bsg.gemm(a, b, sa, sb, **kw)
    monkeypatch.undo()
    assert torch.equal(bsg.gemm(a, b, sa, sb, **kw), slow)
    # what the C++ code leaves to the Python code: given outputs, views, other types
    fast = bsg._marshal()
    x, w = randn(gen, 64, 64), randn(gen, 64)
    for bad in (x.t(), x[0], x.half(), x.cpu(), None, 3, x[:0]):
        assert fast.norm(bad, w, None, 1e-6, 128, 0) is None
    assert fast.norm(x, w[:3], None, 1e-6, 128, 0) is None and fast.norm(x, w, x[:3], 1e-6, 128, 0) is None
    assert fast.norm(x, w, None, "eps", 128, 0) is None and fast.norm(x, w, None, 1e-6, 100, 0) is None
    assert fast.norm(x, w, None, -1.0, 128, 0) == 1      # a status of the library's
    assert fast.act(x, 0, 128, 0) == 1 and fast.act_backward(x, x, 0, 128, 0, True) is None
    assert fast.norm_backward(x, x, w, w.double(), None) is None
    assert fast.gemm(0, 128, x, x, w, w, None, 0, False, None) is None


def test_a_captured_residual_gemm_outlives_the_growth_of_its_workspace():
    """A stream-K call's graph, replayed after a larger call on its stream has taken a larger workspace."""
    gen = gen_of(18)
    bsg.release_workspaces()
    a, b, sa, sb, _, _ = gemm_inputs(gen, 1, 2048, 4096, "nt", 128)
    res = randn(gen, 1, 2048, dtype=torch.bfloat16)
    assert bsg.make_plan(1, 2048, 4096, 128)["sk_ctas"] > 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = bsg.gemm(a, b, sa, sb, residual=res)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = bsg.gemm(a, b, sa, sb, residual=res)
        big = gemm_inputs(gen, 128, 7168, 7168, "nt", 128)[:4]
        first = bsg.gemm(*big)
        for _ in range(20):
            g.replay()
            again = bsg.gemm(*big)
        s.synchronize()
    assert torch.equal(out, want) and torch.equal(first, again)
    bsg.release_workspaces()
    assert bsg.get_last_device_status() == 0


FRESH_CAPTURE = """
import torch
import fp8_block_scaled_bsgemm_b200 as bsg
x = torch.randn(300, 528, device="cuda").bfloat16()
w = torch.ones(528, device="cuda")
rstd = torch.ones(300, device="cuda")
g = torch.cuda.CUDAGraph()
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
with torch.cuda.graph(g, stream=s):
    outs = []
    for gran in (64, 256):
        outs += bsg.rms_norm_quantize(x, w, residual=x, gran=gran, return_rstd=True)
        outs += bsg.rms_norm_quantize(x[:3], w, gran=gran, return_rstd=True)[:2]
        outs += bsg.activation_quantize(x, "gelu", gran=gran)
        outs += bsg.activation_backward_quantize(x, x, "relu", gran=gran)
    outs += bsg.rms_norm_backward(x, x, w, rstd)
g.replay()
torch.cuda.synchronize()
got = [o.clone() for o in outs]
want = []
for gran in (64, 256):
    want += bsg.rms_norm_quantize(x, w, residual=x, gran=gran, return_rstd=True)
    want += bsg.rms_norm_quantize(x[:3], w, gran=gran, return_rstd=True)[:2]
    want += bsg.activation_quantize(x, "gelu", gran=gran)
    want += bsg.activation_backward_quantize(x, x, "relu", gran=gran)
want += bsg.rms_norm_backward(x, x, w, rstd)
assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
print("ok")
"""


def test_the_first_call_of_a_process_can_be_a_captured_one():
    """No call before the capture: set-up of the kernels happens inside it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FRESH_CAPTURE], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


def test_offsets_past_32_bits():
    """More than 2^32 elements: the last rows as if they stood alone, and the sums over all rows."""
    rows, cols, g = 131_200, 32_768, 128
    assert rows * cols > 1 << 32
    gen = gen_of(16)
    bf = torch.bfloat16
    block = randn(gen, g, cols, dtype=bf)            # every row block the same, but for the last one
    tail = randn(gen, g, cols, dtype=bf)
    x = block.repeat(rows // g, 1)
    x[-g:] = tail
    w = randn(gen, cols)
    want = bsg.rms_norm_quantize(tail, w, residual=tail, return_rstd=True)
    q, s, h, rstd = bsg.rms_norm_quantize(x, w, residual=x, residual_out=x, return_rstd=True)
    assert h is x
    for got, alone in ((q, want[0]), (s, want[1]), (x, want[2]), (rstd, want[3])):
        n = alone.shape[0]
        # a row alone is summed by more threads: rstd may differ in its last places, and codes next to a border with it
        if got is x:
            assert torch.equal(got[-n:], alone)
        else:
            a, b = got[-n:].view(torch.uint8).float(), alone.view(torch.uint8).float()
            assert ((a != b).float().mean() < 1e-3) if got is q else torch.allclose(got[-n:], alone, rtol=1e-5)
    del q, s
    dy = x.clone()
    dx, dw = bsg.rms_norm_backward(dy, x, w, rstd, dx=dy)
    assert dx is dy
    check_norm_backward(want[2], want[2], w, rstd[-g:], None, dx[-g:],
                        su.norm_backward(want[2], want[2], w, rstd[-g:])[1].float())
    head = su.norm_backward(su.stream(block, block), su.stream(block, block), w, rstd[:g])[1]
    last = su.norm_backward(want[2], want[2], w, rstd[-g:])[1]
    total = head * (rows // g - 1) + last
    n = su.stream(block, block).double()
    mag = (n * n * rstd[:g].double()[:, None]).abs().sum(0) * (rows // g)
    assert ((dw.double() - total).abs() <= mag * (rows / 100 + 700) * su.U).all()
    del dx, dy, x, h
    torch.cuda.empty_cache()
    z = block.repeat(rows // g, 1)
    z[-g:] = tail
    q, s = bsg.activation_quantize(z, "gelu")
    alone = bsg.activation_quantize(tail, "gelu")
    assert torch.equal(q[-g:], alone[0]) and torch.equal(s[-1:], alone[1])
    del q, s
    q, s, db = bsg.activation_backward_quantize(z, z, "relu")
    alone = bsg.activation_backward_quantize(tail, tail, "relu")
    assert torch.equal(q[-g:], alone[0]) and torch.equal(s[-1:], alone[1])
    sums = block.double().clamp(min=0).sum(0) * (rows // g - 1) + tail.double().clamp(min=0).sum(0)
    assert ((db.double() - sums).abs() <= sums * (g + rows // g) * su.U).all()


def test_scales_are_correctly_rounded_quotients():
    """amax / FMAX by the corrected product: bit for bit the division, over a binade and a range of exponents."""
    for fmt in ("e4m3", "e5m2"):
        mant = torch.arange(1 << 18, device="cuda", dtype=torch.int64) * 32 + 7
        for exponent in (-100, -40, 0, 40, 100, 126):
            v = torch.ldexp(1.0 + mant.double() / (1 << 23), torch.tensor(exponent, device="cuda")).float()
            x = torch.zeros(v.numel(), 16, device="cuda")
            x[:, 3] = v
            x = x.view(1, -1)                      # one row: a block is 64 columns, 4 values
            q, s, _ = bsg.activation_backward_quantize(x.view(-1, 1 << 16), None, gran=64, fmt=fmt, bias_grad=False)
            # (divided on the CPU: torch's CUDA kernel multiplies by the reciprocal of a scalar divisor)
            want = (su.block_amax(x.view(-1, 1 << 16), 64).cpu() / su.FMAX[fmt]).cuda()
            assert want.dtype == torch.float32
            want = torch.where(want > 0, want, torch.ones_like(want))
            assert torch.equal(s, want)


# ------------------------------------------------------------------ a sublayer


@pytest.mark.parametrize("tokens", [1, 300])
def test_sublayer_forward_and_backward(tokens):
    """Norm, product, activation, product into the residual stream, and every gradient, each step against 64 bits on
    the codes that the step before it made."""
    H, F, g = 528, 1552, 128
    gen = gen_of(13, tokens)
    bf = torch.bfloat16
    x, r = randn(gen, tokens, H, dtype=bf), randn(gen, tokens, H, dtype=bf)
    w = 1 + 0.2 * randn(gen, H)
    w1, w2 = randn(gen, F, H, scale=0.05), randn(gen, H, F, scale=0.05)
    b1, b2 = randn(gen, F, scale=0.1), randn(gen, H, scale=0.1)
    q1, s1 = bsg.quantize(w1, g)
    q2, s2 = bsg.quantize(w2, g)
    # forward
    qa, sa, h, rstd = bsg.rms_norm_quantize(x, w, residual=r, eps=EPS, return_rstd=True)
    check_norm(x, w, r, g, "e4m3", (qa, sa, h, rstd))
    z = bsg.gemm(qa, q1, sa, s1, bias=b1)
    qh, sh = bsg.activation_quantize(z, "gelu")
    su.check_codes(qh, sh, su.act(z, "gelu"), g, "e4m3", 2 * su.U, su.gelu_abs(z))
    out = bsg.gemm(qh, q2, sh, s2, bias=b2, residual=h)
    A, W1 = su.dequantize(qa, sa, g, "e4m3"), su.dequantize(q1, s1, g, "e4m3")
    Hd, W2 = su.dequantize(qh, sh, g, "e4m3"), su.dequantize(q2, s2, g, "e4m3")
    check_gemm(out, Hd, W2, b2, None, h)
    # backward
    dout = randn(gen, tokens, H, dtype=bf, scale=0.01)
    qo, so, db2 = bsg.activation_backward_quantize(dout, None, fmt="e5m2")
    su.check_codes(qo, so, dout.double(), g, "e5m2", 0.0)
    dact = bsg.gemm(qo, q2, so, s2.t().contiguous(), layout="nn", a_format="e5m2")   # dout W2: scales by logical block
    D = su.dequantize(qo, so, g, "e5m2")
    check_gemm(dact, D, W2.t(), None, None, torch.zeros_like(dact))
    qz, sz, db1 = bsg.activation_backward_quantize(dact, z, "gelu", fmt="e5m2")
    dz = dact.double() * su.act_slope(z, "gelu")
    extra = dact.double().abs() * su.gelu_slope_abs(z)
    su.check_codes(qz, sz, dz, g, "e5m2", 3 * su.U, extra)
    assert ((db1.double() - dz.sum(0)).abs() <= dz.abs().sum(0) * 400 * su.U + extra.sum(0)).all()
    dy = bsg.gemm(qz, q1, sz, s1.t().contiguous(), layout="nn", a_format="e5m2")     # dz W1
    dx, dw = bsg.rms_norm_backward(dy, h, w, rstd, dresidual=dout)
    check_norm_backward(dy, h, w, rstd, dout, dx, dw)
    # the weight's gradient reads the same codes transposed: dW1 = dz^T A
    dw1 = bsg.gemm(qz, qa, sz.t().contiguous(), sa.t().contiguous(), layout="tn", a_format="e5m2", out_dtype=torch.float32)
    check_gemm(dw1, su.dequantize(qz, sz, g, "e5m2").t(), A.t(), None, None, torch.zeros_like(dw1))
    assert bsg.get_last_device_status() == 0
