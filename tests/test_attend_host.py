"""Host arithmetic of attention's calls (csrc/lb_pages.h) on the CPU, under sanitizers: how the workspace grows."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FLAGS = ["-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror"]


def native(tmp_path, name, *args):
    """What tests/native/<name>.cpp prints."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / name)
    r = subprocess.run([cxx, *FLAGS, os.path.join(ROOT, "tests", "native", name + ".cpp"), "-o", exe],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
    r = subprocess.run([exe, *map(str, args)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    return r.stdout


def test_growing_lengths_keep_little(tmp_path):
    """Outgrown workspaces are kept for captured graphs: all of them together stay below twice the last."""
    allocations, kept = map(int, native(tmp_path, "workspace_check").split())
    assert 1 < allocations <= 12 and 0 < kept < 200
