"""The operators around the GEMM, checked without a GPU: refusals, workspace sizes, launch registers."""
import ctypes
import glob
import os
import re

import pytest
import torch

import fp8_block_scaled_bsgemm_b200 as bsg
from fp8_block_scaled_bsgemm_b200 import build as bsg_build

import sublayer_util as su

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, GRAN, MISALIGNED = 1, 2, 3
MB = 1 << 20   # stand-in addresses, far apart; nothing is dereferenced


def test_residual_gemm_refusals():
    L = bsg.lib()

    def call(residual=3 * MB, out=4 * MB, epi=None, M=64, N=64, K=64, gran=128):
        return L.bsgemm_fp8_gemm_residual(0, 0, 0, MB, 2 * MB, 16, 16, epi, residual, out, M, N, K, gran, None, None)

    assert call(residual=None) == INVALID
    assert call(residual=3 * MB + 8) == MISALIGNED
    assert call(gran=96) == GRAN
    assert call(N=60) == MISALIGNED
    # overlapping, but not the same buffer: 64 x 64 BF16 is 8192 bytes, FP32 twice that
    assert call(residual=4 * MB + 16) == INVALID
    assert call(residual=4 * MB - 8192 + 16) == INVALID
    f32 = bsg.Epilogue(None, 0, 1)
    assert call(residual=4 * MB - 16384 + 16, epi=ctypes.byref(f32)) == INVALID


def _norm(L, x=MB, residual=2 * MB, weight=3 * MB, eps=1e-6, rows=64, cols=64, gran=128, h=4 * MB, q=5 * MB,
          scales=6 * MB, rstd=7 * MB, src=1, wdt=1, fmt=0):
    return L.bsgemm_rms_norm_quantize_fp8(src, wdt, fmt, x, residual, weight, eps, rows, cols, gran, h, q, scales, rstd, None)


@pytest.mark.parametrize("change,want", [
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(q=None), INVALID), (dict(scales=None), INVALID),
    (dict(residual=None), INVALID), (dict(h=None), INVALID),             # both or neither
    (dict(src=2), INVALID), (dict(wdt=-1), INVALID), (dict(fmt=2), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(rows=-3), INVALID), (dict(rows=(1 << 30) + 1), INVALID), (dict(cols=(1 << 24) + 16), INVALID), (dict(rstd=None), INVALID),
    (dict(gran=32), GRAN), (dict(cols=72), MISALIGNED), (dict(x=MB + 8), MISALIGNED), (dict(weight=3 * MB + 4), MISALIGNED),
    (dict(q=5 * MB + 8), MISALIGNED), (dict(scales=6 * MB + 2), MISALIGNED), (dict(rstd=7 * MB + 1), MISALIGNED),
    (dict(h=MB + 16), INVALID), (dict(h=2 * MB - 16), INVALID),          # a shifted part of an input
    (dict(q=MB), INVALID), (dict(q=4 * MB), INVALID), (dict(scales=3 * MB), INVALID), (dict(rstd=6 * MB), INVALID),
    (dict(h=3 * MB - 8192 + 16), INVALID),
])
def test_norm_refusals(change, want):
    assert _norm(bsg.lib(), **change) == want


def _norm_bwd(L, dy=MB, h=2 * MB, weight=3 * MB, rstd=4 * MB, skip=5 * MB, rows=64, cols=64, dx=6 * MB, dw=7 * MB,
              ws=8 * MB, nbytes=None, src=1, wdt=1):
    need = L.bsgemm_rms_norm_backward_workspace(rows, cols)
    return L.bsgemm_rms_norm_backward(src, wdt, dy, h, weight, rstd, skip, rows, cols, dx, dw, ws,
                                      need if nbytes is None else need + nbytes, None)


@pytest.mark.parametrize("change,want", [
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(weight=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dx=None), INVALID), (dict(dw=None), INVALID), (dict(ws=None), INVALID), (dict(nbytes=-1), INVALID),
    (dict(src=5), INVALID), (dict(wdt=2), INVALID), (dict(rows=0), INVALID), (dict(cols=65536 + 16), INVALID),
    (dict(cols=24), MISALIGNED), (dict(dy=MB + 8), MISALIGNED), (dict(skip=5 * MB + 2), MISALIGNED),
    (dict(dw=7 * MB + 4), MISALIGNED), (dict(ws=8 * MB + 8), MISALIGNED), (dict(rstd=4 * MB + 1), MISALIGNED),
    (dict(dx=2 * MB), INVALID), (dict(dx=MB + 16), INVALID), (dict(dw=6 * MB), INVALID), (dict(ws=6 * MB), INVALID),
    (dict(dw=3 * MB), INVALID),
])
def test_norm_backward_refusals(change, want):
    assert _norm_bwd(bsg.lib(), **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(z=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(act=0), INVALID), (dict(act=3), INVALID),
    (dict(src=2), INVALID), (dict(fmt=4), INVALID), (dict(rows=0), INVALID), (dict(gran=100), GRAN), (dict(cols=40), MISALIGNED),
    (dict(z=MB + 4), MISALIGNED), (dict(q=2 * MB + 8), MISALIGNED), (dict(s=3 * MB + 2), MISALIGNED), (dict(q=MB), INVALID),
    (dict(s=MB + 64), INVALID),
])
def test_activation_refusals(change, want):
    a = dict(src=1, fmt=0, act=2, z=MB, rows=64, cols=64, gran=128, q=2 * MB, s=3 * MB) | change
    L = bsg.lib()
    assert L.bsgemm_activation_quantize_fp8(a["src"], a["fmt"], a["act"], a["z"], a["rows"], a["cols"], a["gran"],
                                            a["q"], a["s"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(dout=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(z=None), INVALID),
    (dict(act=0), INVALID),                                              # z without an activation
    (dict(act=5), INVALID), (dict(fmt=-1), INVALID), (dict(ws=None), INVALID), (dict(nbytes=-1), INVALID),
    (dict(gran=1), GRAN), (dict(cols=8), MISALIGNED), (dict(z=2 * MB + 8), MISALIGNED), (dict(db=5 * MB + 2), MISALIGNED),
    (dict(ws=6 * MB + 2), MISALIGNED), (dict(q=MB), INVALID), (dict(q=2 * MB), INVALID), (dict(ws=3 * MB), INVALID),
    (dict(db=4 * MB), INVALID),
])
def test_activation_backward_refusals(change, want):
    a = dict(src=1, fmt=0, act=2, dout=MB, z=2 * MB, rows=300, cols=64, gran=128, q=3 * MB, s=4 * MB, db=5 * MB, ws=6 * MB,
             nbytes=0) | change
    L = bsg.lib()
    need = L.bsgemm_activation_backward_workspace(a["rows"], a["cols"], a["gran"])
    assert L.bsgemm_activation_backward_quantize_fp8(
        a["src"], a["fmt"], a["act"], a["dout"], a["z"], a["rows"], a["cols"], a["gran"], a["q"], a["s"], a["db"], a["ws"],
        max(0, need + a["nbytes"]), None) == want


def test_workspace_sizes():
    L = bsg.lib()
    assert L.bsgemm_rms_norm_backward_workspace(1, 64) == 64 * 4
    assert L.bsgemm_rms_norm_backward_workspace(1 << 20, 4096) == 640 * 4096 * 4
    assert L.bsgemm_rms_norm_backward_workspace(0, 64) == 0
    assert L.bsgemm_activation_backward_workspace(128, 64, 128) == 0      # one row of sums is dbias itself
    assert L.bsgemm_activation_backward_workspace(129, 64, 128) == 2 * 64 * 4
    assert L.bsgemm_activation_backward_workspace(1, 64, 256) == 4 * 64 * 4
    assert L.bsgemm_activation_backward_workspace(1 << 30, 1 << 20, 64) == (1 << 24) * (1 << 20) * 4


def test_epilogue_instances_have_the_planned_launch_registers():
    """The widest tiles' register split needs exactly 168 launch registers, in the epilogue's instances too."""
    bsg_build.build()
    logs = glob.glob(os.path.join(ROOT, "_build", "bsgemm_inst_epi_g*.log"))
    assert len(logs) == 12
    wide = 0
    for log in logs:
        cur = None
        for ln in open(log):
            m = re.search(r"Compiling entry function '_ZN3bsg(?:13bsgemm_kernelILi(\d+)E|18bsgemm_pair_kernel)", ln)
            if m:
                cur = int(m.group(1) or 256)
            elif cur is not None and "Used" in ln:
                regs = int(re.search(r"Used (\d+) registers", ln).group(1))
                assert regs == 168 if cur == 256 else regs <= 168, (log, ln)
                wide += cur == 256
                cur = None
    assert wide == 12 * 3   # split, whole tiles and the CTA pair


def test_binding_refuses_host_tensors_and_wrong_arguments():
    x = torch.zeros((128, 256))
    w = torch.ones(256)
    with pytest.raises(ValueError):
        bsg.rms_norm_quantize(x, w)
    with pytest.raises(ValueError):
        bsg.rms_norm_backward(x, x, w, torch.ones(128))
    with pytest.raises(ValueError):
        bsg.activation_quantize(x, "gelu")
    with pytest.raises(ValueError):
        bsg.activation_backward_quantize(x, x, "gelu")


# ------------------------------------------------------------------ the plain forms themselves


def test_plain_gradients_against_differences():
    """The formulas that the GPU tests hold the kernels to, against central differences in 64 bits."""
    gen = torch.Generator().manual_seed(3)
    h = torch.randn(5, 48, generator=gen, dtype=torch.float64)
    w = 1 + 0.3 * torch.randn(48, generator=gen, dtype=torch.float64)
    dy = torch.randn(5, 48, generator=gen, dtype=torch.float64)
    eps, d = 1e-3, 1e-6

    def loss(h, w):
        return (su.norm(h, w, eps)[0] * dy).sum()

    dx, dw = su.norm_backward(dy, h, w, su.norm(h, w, eps)[1])
    for i, j in [(0, 0), (2, 17), (4, 47)]:
        e = torch.zeros_like(h)
        e[i, j] = d
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - dx[i, j]) < 1e-7
        e = torch.zeros_like(w)
        e[j] = d
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - dw[j]) < 1e-7
    z = torch.tensor([-6.0, -2.5, -0.3, 0.4, 1.7, 5.0], dtype=torch.float64)
    for name in ("relu", "gelu"):
        num = (su.act(z + d, name) - su.act(z - d, name)) / (2 * d)
        assert (num - su.act_slope(z, name)).abs().max() < 1e-8


def test_fitted_gelu():
    """The polynomial that the activation kernels evaluate, in FP32 steps, against 64 bits.

    T = Phi(-u) = 2^P <= 1/2 is off by 1.1e-7 of the fit and by ln 2 T times P's error in FP32, whose terms add up
    to less than 2 |P| + 2 (two roundings of each, 4 U (|P| + 1)): ln 2 T 4 U (|P| + 1) <= 3 U, P being -1 at T = 1/2;
    one more for the exponential. GELU: that times |z|, 1.1e-7 + 4 U = 3.5e-7, and its own rounding. The slope adds
    u phi(u) <= 0.25 with (u^2 / 2 + 4) U of itself, below U, and three sums below 1.2: 5 U more, 6.5e-7.
    """
    src = open(os.path.join(ROOT, "fp8_block_scaled_bsgemm_b200", "csrc", "bsgemm_gelu.cuh")).read()
    num = r"-?[\d.]+(?:e-\d+)?"
    first = float(re.search(rf"t\[i\] = both2\(({num})f\)", src).group(1))
    coef = [float(c.strip().rstrip("f")) for c in re.search(r"coef\[6\] = \{([^}]*)\}", src).group(1).split(",")]
    assert len(coef) == 6
    z = torch.linspace(-20, 20, 800001, dtype=torch.float64).float()
    n = -z.abs().clamp(max=14.0)
    q = torch.full_like(z, first)
    for c in coef:
        q = (q.double() * n.double() + torch.tensor(c).double()).float()
    t = torch.exp2(q)
    gelu = (z.clamp(min=0).double() + t.double() * n.double()).float()
    assert ((gelu.double() - su.act(z, "gelu")).abs() <= (1.1e-7 + 4 * su.U) * z.abs().double() + su.U * gelu.abs().double()).all()
    phi = torch.exp2(((n * n).double() * -0.72134752 - 1.32574807).float())
    h = (n.double() * phi.double() + (t - 0.5).double()).float()
    slope = torch.where(z < 0, h, -h) + 0.5
    assert (slope.double() - su.act_slope(z, "gelu")).abs().max() < 1.1e-7 + 9 * su.U
    # past the clamp nothing is left of the tail
    assert float(t[0]) < 2.0 ** -126
