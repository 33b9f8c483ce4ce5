"""The quantizing arithmetic of the expert-layer kernels, restated in C and checked
exhaustively (tests/native/corrected_quotient_exhaustive.c): the scale amax / 448 by a
corrected product for every BF16 amax in the window and every FP32 mantissa at several
exponents, and the E4M3 code of fl32(x / s) by a reciprocal in two parts for every such amax
against every BF16 x with |x| <= amax, the approximation of 1/s up to two units off."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_corrected_quotient_is_exact_for_every_bf16_value_and_scale(tmp_path):
    exe = tmp_path / "corrected_quotient"
    subprocess.run(["gcc", "-O2", "-fopenmp", "-fno-fast-math", "-ffp-contract=off", "-o", str(exe),
                    os.path.join(HERE, "native", "corrected_quotient_exhaustive.c"), "-lm"], check=True)
    p = subprocess.run([str(exe)], capture_output=True, text=True, timeout=1200)
    assert p.returncode == 0 and p.stdout.strip().endswith("mismatches 0"), p.stdout[-2000:]
