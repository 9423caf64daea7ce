"""The sharing out of attention over a paged cache, on the host (tests/paged_schedule.cpp): every tile
of every unit is taken by exactly one of the workers, of which there may be one or many, with
and without units side by side."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT
from test_c_abi_caller import _cuda_home


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx, cuda = shutil.which("g++"), _cuda_home()
    if not cxx or not cuda:
        pytest.skip("no C++ compiler or CUDA headers")
    exe = str(tmp_path_factory.mktemp("schedule") / "paged_schedule")
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Wno-unused-function", "-I", os.path.join(cuda, "include"),
                        os.path.join(ROOT, "tests", "paged_schedule.cpp"), "-o", exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return exe


@pytest.mark.parametrize("seed", range(6))
def test_every_tile_is_taken_once(program, seed):
    r = subprocess.run([program, str(seed), "150"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
