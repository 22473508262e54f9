"""Which copies a block waits for after a bounded wait has run out, checked on
the host: tests/native/ring_drain_check.cu includes the header that the kernels
use."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT


def test_no_copy_is_left_in_flight(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = tmp_path / "ring_drain_check"
    src = os.path.join(ROOT, "tests", "native", "ring_drain_check.cu")
    inc = os.path.join(ROOT, "latent_attention_b200", "csrc")
    subprocess.run([nvcc, "-std=c++17", "-O2", "-Wno-deprecated-gpu-targets", "-o", str(exe), src,
                    "-I", inc], check=True, capture_output=True, text=True, timeout=300)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    assert out.stdout.startswith("ok ")
