"""The rotary append divides fp32 keys by scales of fp32 maxima with the append kernels'
reciprocal product and one correction.  This test builds tests/cuda/quant_fp32.cu and checks,
on the GPU, that the e4m3 codes equal those of CUDA's correctly rounded quotient wherever they
could differ: for every mantissa of a scale, around every border between two codes."""
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_fp32_division_matches_ieee_around_every_border(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    exe = str(tmp_path / "quant_fp32")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17",
                    "-I", os.path.join(ROOT, "paged_fp8_kv_append_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "cuda", "quant_fp32.cu"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    print(r.stdout)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "mismatches=0" in r.stdout
