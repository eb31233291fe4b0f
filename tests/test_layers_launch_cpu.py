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


def test_small_norms_stay_in_the_caches_for_the_products_that_read_them(tmp_path):
    """The rule of layers_sizes.h at both sides of its bound, and that of the loads of large calls."""
    if shutil.which("g++") is None:
        pytest.skip("g++ is missing")
    src, exe = tmp_path / "rules.cpp", tmp_path / "rules"
    src.write_text('#include "layers_sizes.h"\n#include <cstdio>\nint main() {\n'
                   'const int64_t rows[] = {1, 333, 1000, 2048, 16384};\n'
                   'for (int64_t r : rows) std::printf("%d %d\\n", opt8::stays(r * 4096 * 2), opt8::streams(r * 4096 * 6)); }\n')
    subprocess.run(["g++", "-std=c++17", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert out.split() == "1 0 1 0 1 0 0 0 0 1".split()
