"""The quotient that the norm and activation kernels encode, beside every border between FP8 codes.

``tests/block_quotient_model.c`` runs the steps of ``bsgr::quotients`` (csrc/bsgemm_rows.cuh) in IEEE single
precision for every mantissa of the scale, with every value near the product of the scale and a border.
"""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_quotient_matches_division_beside_every_border(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    exe = str(tmp_path / "block_quotient_model")
    flags = ["-O2", "-ffp-contract=off", "-std=c99"]
    src = os.path.join(HERE, "block_quotient_model.c")
    if subprocess.run([cc, *flags, "-fopenmp", src, "-o", exe, "-lm"], capture_output=True).returncode != 0:
        subprocess.run([cc, *flags, src, "-o", exe, "-lm"], check=True, capture_output=True)   # no OpenMP: one thread
    run = subprocess.run([exe, "1"], capture_output=True, text=True, timeout=900)
    assert run.returncode == 0, run.stdout + run.stderr
    pairs, differ, wrong = map(int, re.search(r"(\d+) pairs, (\d+) differ; .* border (\d+) times", run.stdout).groups())
    assert pairs == (1 << 23) * 16 * 9 and differ == 0 and wrong > 0


def test_the_kernels_take_the_modelled_steps():
    """The encoder's source has the model's three steps, and no code is made from an uncorrected product."""
    root = os.path.join(os.path.dirname(HERE), "fp8_block_scaled_bsgemm_b200", "csrc")
    rows = open(os.path.join(root, "bsgemm_rows.cuh")).read()
    assert "__frcp_rn(r.s)" in rows and "rcp.approx" not in rows
    body = re.search(r"void quotients\(.*?\n}\n", rows, re.S).group(0)
    assert re.search(r"p = mul2\(v\[i\], nr\);\s*"
                     r"v\[i\] = bsg::ffma2\(bsg::ffma2\(p, both\(s\.s\), v\[i\]\), nr, p\);", body)
    blocks = open(os.path.join(root, "bsgemm_blocks.cuh")).read()
    assert "mul2(v[j][i], both(s.rcp))" not in blocks
