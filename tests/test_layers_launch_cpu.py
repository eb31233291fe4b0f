"""What the host code of opt8_layers.h passes on to the kernels (tests/layers_launch/driver.cpp):
nothing that its checks left out.  On the CPU, with stand-ins for the launches."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "precision_optimizer_step_amd", "csrc")
ROCM_INCLUDE = "/opt/rocm/include"


def test_unchecked_pointers_do_not_reach_a_kernel(tmp_path):
    if shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE):
        pytest.skip("g++ or the ROCm headers are missing")
    exe = tmp_path / "launch_driver"
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I" + ROCM_INCLUDE, "-I" + CSRC, os.path.join(CSRC, "layers_host.cpp"),
                    os.path.join(ROOT, "tests", "layers_launch", "driver.cpp"), "-o", str(exe)], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0 and "all checks passed" in run.stdout, run.stdout
