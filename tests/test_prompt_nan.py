"""Where the prompt kernel looks for NaN values, checked without a GPU:
tests/host/prompt_nan_check.cu includes the kernel's source and compares its index
arithmetic with counting, under the compiler's check for signed overflow (the state in
which no NaN has been met is a range from the largest integer to -1)."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_attention_52_gb300", "csrc")


def test_index_arithmetic(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "prompt_nan_check")
    # device code as PTX only (no GPU code generation needed: nothing is launched)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=compute_103a",
                    "--expt-relaxed-constexpr", "-Xcompiler", "-fsanitize=signed-integer-overflow,-fno-sanitize-recover",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "host", "prompt_nan_check.cu"),
                    os.path.join(CSRC, "attn_cache.cu"), "-o", exe], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "bad 0" in r.stdout
