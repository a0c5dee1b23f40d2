"""Plain 64-bit forms of the operators around the GEMM, and their tolerances (not a test module).

U = 2^-24 is FP32's largest relative rounding. A sum of terms added in FP32 to
depth d (the longest chain of additions any term passes through) is off by at
most d U times the sum of the terms' magnitudes, first order; products and
quotients add one U each. Every bound below counts those, and each output's own
rounding once: BF16 2^-8, FP32 U, FP8 half a step.
"""
import math

import torch

U = 2.0 ** -24
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
MANTISSA = {"e4m3": 3, "e5m2": 2}      # stored bits
MIN_EXP = {"e4m3": -6, "e5m2": -14}    # of the smallest normal value


def half_step(v, fmt):
    """Half the distance between FP8 neighbours at magnitude |v|."""
    _, e = torch.frexp(v.abs())           # |v| = m 2^e, m in [1/2, 1)
    e = torch.clamp(torch.where(v == 0, torch.full_like(e, -1000), e - 1), min=MIN_EXP[fmt])
    return torch.exp2((e - MANTISSA[fmt] - 1).double())


def out_rounding(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def block_amax(y, g):
    rows, cols = y.shape
    rb, cb = -(-rows // g), -(-cols // g)
    t = torch.zeros(rb * g, cb * g, dtype=y.dtype, device=y.device)
    t[:rows, :cols] = y.abs()
    return t.view(rb, g, cb, g).amax(dim=(1, 3))


def spread(s, g, rows, cols):
    """A value per block at each of the block's elements."""
    return s.repeat_interleave(g, 0)[:rows].repeat_interleave(g, 1)[:, :cols]


def check_codes(q, scales, y, g, fmt, rel, absolute=None):
    """q, scales against the 64-bit y, computed in FP32 to within rel |y| + absolute.

    A scale is the amax over FMAX: off by rel (and one rounding) of itself, plus
    the largest absolute part in the block. A code's quotient is off by the
    value's part, the scale's part and two roundings (the reciprocal and the
    product), before the rounding to FP8, half a step at either neighbour.
    """
    rows, cols = y.shape
    amax = block_amax(y, g)
    want = amax / FMAX[fmt]
    want = torch.where(want > 0, want, torch.ones_like(want))
    a = torch.zeros_like(y) if absolute is None else absolute
    s_tol = want * (rel + 2 * U) + block_amax(a, g) / FMAX[fmt] * (amax > 0)
    got_s = scales.double().view_as(want)
    # scales are whole multiples of FP32's smallest step where they are tiny
    assert ((got_s - want).abs() <= s_tol + 2.0 ** -149).all(), float(((got_s - want).abs() / (s_tol + 2.0 ** -149)).max())
    s = spread(got_s, g, rows, cols)
    v = y / s
    got = q.view(rows, cols).view(FP8[fmt]).double()
    assert torch.isfinite(got).all() or not torch.isfinite(y).all()
    clipped = v.clamp(-FMAX[fmt], FMAX[fmt])
    tol = torch.maximum(half_step(clipped, fmt), half_step(got, fmt)) * 1.0 + v.abs() * (rel + 3 * U) + a / s
    bad = ~((got - clipped).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), v[bad][:4].tolist())


# ------------------------------------------------------------------ formulas


def stream(x, residual):
    return x if residual is None else (x.double() + residual.double()).to(x.dtype)


def norm(h, weight, eps):
    h = h.double()
    rstd = (h.square().mean(1) + eps).rsqrt()
    return h * rstd[:, None] * weight.double(), rstd


def norm_backward(dy, h, weight, rstd, skip=None):
    dy, h, w, r = dy.double(), h.double(), weight.double(), rstd.double()[:, None]
    n = h * r
    dn = dy * w
    dx = r * (dn - n * (dn * n).mean(1, keepdim=True))
    if skip is not None:
        dx = dx + skip.double()
    return dx, (dy * n).sum(0)


def phi(z):
    return torch.special.ndtr(z)


def act(z, name):
    z = z.double()
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * phi(z)
    return z


def act_slope(z, name):
    if name in (None, "none"):
        return 1.0
    z = z.double()
    if name == "relu":
        return (z > 0).double()
    return phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def dequantize(q, scales, g, fmt):
    rows, cols = q.shape
    return q.view(FP8[fmt]).double() * spread(scales.double(), g, rows, cols)


# ------------------------------------------------------------------ bounds


def rstd_rel(cols, g):
    """Relative bound of the forward call's rstd: the sum of squares' (all terms positive), halved, and the tail's.

    A thread adds a run's 8 squares pairwise (5 roundings) into its row's sum,
    over its share of the column blocks (at least 1/16 of them in the largest
    cluster, all of them in the smallest, which has at most one); 5 exchanges in
    the warp, up to 31 block slots and 16 CTAs follow, then the mean, eps and
    the reciprocal root.
    """
    blocks = -(-cols // g)
    return (5 + -(-blocks // 16) + 1 + 5 + 31 + 16 + 2) / 2 * U + 2 * U


def gelu_abs(z):
    """FP32 bound of z Phi(z) beside its own rounding: the fitted tail's (tests/test_sublayer_host.py has its parts)."""
    return (1.1e-7 + 4 * U) * z.abs().double()


def gelu_slope_abs(z):
    """The same for Phi(z) + z phi(z)."""
    return torch.full_like(z, 1.1e-7 + 9 * U, dtype=torch.float64)
