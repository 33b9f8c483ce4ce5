"""The E4M3 conversion of the activation checkpoint, restated in C and checked for every
pair it can meet (tests/native/corrected_quotient_exhaustive.c): every BF16 group maximum
whose scale s = fl32(amax / 448) lies in [2^-100, 2^100] against every BF16 x with
|x| <= amax, about 8.9e8 pairs.  The corrected quotient's code must equal
E4M3(fl32(x / s)) in every case."""
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
