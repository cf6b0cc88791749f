"""The order in which attention's many-row kernel fills and reads its LDS (csrc/lb_pages.h) on the CPU, under sanitizers:
between two barriers nothing is written that a slower wave may still read."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FLAGS = ["-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror"]


def test_nothing_is_overwritten(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "tiles_check")
    r = subprocess.run([cxx, *FLAGS, os.path.join(ROOT, "tests", "native", "tiles_check.cpp"), "-o", exe],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) > 3000
