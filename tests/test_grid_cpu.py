"""Host-side check that the optimizer's launches of any number of chunks are ones that HIP takes (csrc/grid.h,
compiled with the host compiler)."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def test_launches_of_any_number_of_chunks(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "check")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", os.path.join(HERE, "grid_check.cpp"), "-o", exe], check=True)
    # a chunk is 1024 values, a set holds up to 2^37 in up to 2^20 tensors
    counts = [0, 1, 2, 132648, 2 ** 27 + 2 ** 20, 2 ** 31 - 1] + [3 ** k for k in range(1, 19)] + \
        [2 ** k + d for k in range(17, 31) for d in (-1, 0, 1)]
    p = subprocess.run([exe], input="\n".join(map(str, counts)), capture_output=True, text=True)
    assert p.returncode == 0 and p.stdout.split() == ["ok", str(len(counts))], p.stdout


def test_optimizer_launches_go_through_it():
    """No launch of the optimizer's puts a whole set's chunks along x."""
    src = open(os.path.join(os.path.dirname(HERE), "orthogonal_reparameterized_poetx_amd", "csrc", "optim.hip")).read()
    assert src.count(" launches(") == 2 and "dim3 grid((unsigned)set->chunks)" not in src
