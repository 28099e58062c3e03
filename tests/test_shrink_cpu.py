"""Host-side check of the LDS layout of the adapters' shrink: the functions of
csrc/shrink.h, compiled with the host compiler; tests/shrink_check.cpp goes
through every group of ranks that a workgroup may get."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join("orthogonal_reparameterized_poetx_amd", "csrc")


def _run(root, exe):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    subprocess.run([cxx, "-std=c++17", "-O2", "-Wall", os.path.join(root, "tests", "shrink_check.cpp"), "-o", exe],
                   check=True)
    return subprocess.run([exe], capture_output=True, text=True)


def test_groups_of_ranks_stay_inside_the_lds(tmp_path):
    p = _run(os.path.dirname(HERE), str(tmp_path / "check"))
    assert p.returncode == 0 and p.stdout.startswith("ok"), p.stdout + p.stderr


def test_check_catches_groups_in_the_padding(tmp_path):
    """A copy whose groups in the padding have no ranks less (zero or negative pieces, which the kernel divides by)."""
    d = tmp_path / CSRC
    d.mkdir(parents=True)
    hdr = open(os.path.join(os.path.dirname(HERE), CSRC, "shrink.h")).read()
    old = "left < 0 ? 0 : left < 16 * rt"
    assert old in hdr
    (d / "shrink.h").write_text(hdr.replace(old, "left < 16 * rt"))
    (tmp_path / "tests").mkdir()
    (tmp_path / "tests" / "shrink_check.cpp").write_text(open(os.path.join(HERE, "shrink_check.cpp")).read())
    p = _run(str(tmp_path), str(tmp_path / "check"))
    assert p.returncode == 1 and "FAIL" in p.stdout
