"""Which kernel each size runs in (products_choice.h, compiled here without a GPU): the sizes of
the GPU tests reach every kernel, and no launch has more threads than HIP takes."""

import os
import shutil
import subprocess

import pytest

import products_shapes as shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is missing")
    exe = tmp_path_factory.mktemp("choice") / "choice"
    cmd = ["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
           "-I" + os.path.join(ROOT, "precision_optimizer_step_amd", "csrc"),
           os.path.join(ROOT, "tests", "products_choice", "driver.cpp"), "-o", str(exe)]
    subprocess.run(cmd, check=True)

    def run(lines):
        out = subprocess.run([str(exe)], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True).stdout
        return [[int(v) for v in line.split()] for line in out.splitlines()]
    return run


@pytest.mark.parametrize("tile", [0, 1])
def test_products_reach_every_tiling(ask, tile):
    got = ask([f"fp8 {m} {n} {k} {tile}" for (m, n, k), _ in shapes.PRODUCTS])
    assert got == [[t] for _, t in shapes.PRODUCTS]
    assert {t for _, t in shapes.PRODUCTS} == {-1, 0, 1, 2, 3, 4}


def test_gated_block_reaches_every_tiling(ask):
    got = ask(["gated %d %d %d" % s[0] for s in shapes.GATED])
    assert got == [list(s[1:]) for s in shapes.GATED]
    assert {s[1] for s in shapes.GATED} == {-1, 0, 1, 2, 3, 4}
    assert {s[2] for s in shapes.GATED} == {s[3] for s in shapes.GATED} == {0, 1, 2, 3, 4}
    assert any(s[4] > 1 for s in shapes.GATED)


def test_depths_of_the_kernels_for_few_rows():
    """By the loops' own arithmetic: a wave takes steps s*w/4 to s*(w+1)/4, four at a time."""
    for depths, size in ((shapes.FEW_GATED_D, 2), (shapes.FEW_PRODUCT_K, 1)):
        fours, singles, tails = set(), set(), set()
        for d in depths:
            steps = d * size // 128
            for w in range(4):
                n = steps * (w + 1) // 4 - steps * w // 4
                fours.add(n // 4)
                singles.add(n % 4)
            tails.add(d * size % 128 != 0)
        assert {0, 1} <= fours and max(fours) >= 4 and {0, 3} <= singles and tails == {False, True}


def test_no_launch_has_too_many_threads(ask):
    """HIP takes fewer than 2^32 threads in a launch: sizes at and beside the powers of two up to
    the documented limits stay below."""
    (worst,), = ask(["grids"])
    assert 2 ** 30 < worst < 2 ** 32
