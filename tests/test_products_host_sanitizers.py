"""The operators' host code (checks and entry points) under AddressSanitizer and UBSan, on the
CPU: random arguments against a byte-by-byte check of overlaps, sizes at their limits, a failed
launch (tests/products_sanitize/driver.cpp).  No GPU code is built here."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "products_sanitize")
CSRC = os.path.join(ROOT, "precision_optimizer_step_amd", "csrc")
ROCM_INCLUDE = "/opt/rocm/include"


def test_host_code_is_clean_under_sanitizers(tmp_path):
    if shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("g++ or the ROCm headers are missing")
    exe = tmp_path / "products_driver"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=" + "address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I" + ROCM_INCLUDE, "-I" + CSRC,
           os.path.join(CSRC, "products_host.cpp"), os.path.join(HERE, "driver.cpp"), "-o", str(exe)]
    build = subprocess.run(cmd, capture_output=True, text=True)
    if build.returncode != 0 and "san" in build.stderr.lower() and "cannot find" in build.stderr.lower():
        pytest.skip("sanitizer runtime not installed")
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, (run.stdout[-4000:], run.stderr[-4000:])
    assert "all checks passed" in run.stdout, run.stdout
