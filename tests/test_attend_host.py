"""Host arithmetic of attention's calls (csrc/lb_pages.h) on the CPU, under sanitizers: how the workspace grows, and which
calls have which tiles."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests import attendcases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FLAGS = ["-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror"]


def native(tmp_path, name, *args):
    """What tests/native/<name>.cpp prints."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / name)
    if not os.path.exists(exe):
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


def test_calls_of_wide_tiles(tmp_path):
    """The calls of test_gpu_attend_wide_tiles have tiles of 256 rows, not cut, for every padded width up to 128."""
    widths = set()
    for name, kw in attendcases.WIDE.items():
        c = attendcases.wide(np.random.default_rng(0), **kw)
        for window in (0, 1, 37, 48, 60, 150):
            args = attendcases.plan_arguments(c, window)
            assert native(tmp_path, "plan_print", *args).split()[:2] == ["256", "1"], (name, window)
        widths.add(args[1])
    assert widths == {32, 64, 96, 128}
