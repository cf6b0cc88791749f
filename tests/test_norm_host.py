"""The shapes in which lb_norm is launched (csrc/lb_norm.h), on the CPU."""
import os
import shutil
import subprocess

import pytest

from tests import normcases

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FLAGS = ["-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Wextra", "-Werror"]


def test_calls_of_every_shape(tmp_path):
    """The calls of test_gpu_norm_shapes are launched as their list says, and a row's pieces hold its columns."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "norm_print")
    r = subprocess.run([cxx, *FLAGS, os.path.join(ROOT, "tests", "native", "norm_print.cpp"), "-o", exe],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout

    def shapes(calls):
        r = subprocess.run([exe, *(str(v) for call in calls for v in call)], stdout=subprocess.PIPE, text=True, timeout=60)
        return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]

    calls = [(rows, width) for _, rows, width in normcases.CALLS]
    assert shapes(calls) == [shape for shape, _, _ in normcases.CALLS]
    calls = [(rows, width) for rows in (1, 255, 256, 2047, 2048, 1 << 20) for width in range(1, 32769, 31)] + [(1, 32768)]
    found = shapes(calls)
    assert all(8 * t * k >= width for (t, k), (_, width) in zip(found, calls))
    assert set(found) == set(normcases.SHAPES)
