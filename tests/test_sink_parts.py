"""The host side of the backward with sinks, checked without a GPU: tests/host/sink_parts_check.cu
includes the backward's source, asks it into how many parts it divides the sink tiles' items
of problems of many shapes on 152 SMs, and checks that items and parts take every step once.
The four shapes that the GPU tests compare as split are split, at both head dimensions."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_attention_52_gb300", "csrc")


def test_parts_take_every_step_once(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "sink_parts_check")
    # device code as PTX only (no GPU code generation needed: nothing is launched)
    subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=compute_103a",
                    "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "host", "sink_parts_check.cu"), "-o", exe],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "bad 0" in r.stdout
