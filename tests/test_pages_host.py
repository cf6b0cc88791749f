"""The work items of the cache calls (csrc/lb_pages.h) on the CPU, under sanitizers: every row and key has its place
exactly once, and nothing that starts, lengths and pages may hold leads outside the arrays."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FLAGS = ["-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror"]


def test_work_items(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "pages_check")
    r = subprocess.run([cxx, *FLAGS, os.path.join(ROOT, "tests", "native", "pages_check.cpp"), "-o", exe],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    calls, rows, pieces = map(int, r.stdout.split())
    assert calls > 200000 and rows > 1000000 and pieces > 100000
