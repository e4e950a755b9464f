"""The epilogues of ragged rows read inside their matrices: the address arithmetic of the kernels
(ragged.hpp) compiled for the host and walked over every tile of many sizes."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "w4a16_group_wise_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_ragged_groups_read_inside_their_matrices(tmp_path):
    exe = tmp_path / "ragged_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-I", CSRC, "-o", str(exe), os.path.join(HERE, "ragged_check.cpp")],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    bad, wrong, caught = (int(v) for v in out.split())
    assert bad == 0 and wrong == 0
    assert caught > 0  # the walk reaches groups wholly past the last row
