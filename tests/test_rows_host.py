"""Whether two strided arrays share memory (csrc/lb_rows.h), on the CPU against marking every byte."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FLAGS = ["-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror"]


def test_strided_arrays(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "rows_check")
    r = subprocess.run([cxx, *FLAGS, os.path.join(ROOT, "tests", "native", "rows_check.cpp"), "-o", exe],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    pairs, shared, cautious, blocks, refused = map(int, r.stdout.split())
    assert pairs > 100000 and shared > 10000 and blocks > 1000
    assert refused == 0, "column blocks of one buffer were refused"
