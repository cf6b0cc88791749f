"""Host arithmetic of attention's calls (csrc/lb_pages.h) on the CPU, under sanitizers: how the workspace grows, and which
calls have which tiles."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from tests import attendcases, cacheref
from tests.attendcases import WINDOWS

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
    """The calls of test_gpu_attend_wide_tiles have tiles of 256 rows, not cut, for every padded width up to 128; with
    fewer rows a sequence, a narrower window or wider heads they would not have them."""
    widths = set()
    for name, kw in attendcases.WIDE.items():
        c = attendcases.wide(np.random.default_rng(0), **kw)
        for window in WINDOWS + (4200,):
            args = attendcases.plan_arguments(c, window)
            assert native(tmp_path, "plan_print", *args).split()[:2] == ["256", "1"], (name, window)
        widths.add(args[1])
    assert widths == {32, 64, 96, 128}
    assert native(tmp_path, "plan_print", *attendcases.plan_arguments(c, 4095)).split()[0] == "128"
    c.dim = 136
    assert native(tmp_path, "plan_print", *attendcases.plan_arguments(c)).split()[0] == "128"
    # a batch with chunks of 600 rows on 33 heads, and a chunk among 127 tokens
    for lengths, new, heads in (([3000] * 16, [600] * 16, 33), ([3000] * 128, [100] + [1] * 127, 8)):
        c = cacheref.Case(np.random.default_rng(0), lengths, new, 64, heads, heads, 128)
        assert native(tmp_path, "plan_print", *attendcases.plan_arguments(c)).split()[0] == "128"


def test_reference_by_products():
    """attendcases.attend is cacheref.attend."""
    rng = np.random.default_rng(2)
    c = cacheref.Case(rng, [60, 1, 33], [25, 1, 33], 16, 2, 4, 24)
    ref = cacheref.Cache(c.pages, 16, 2, 24)
    start = np.array([0, 60, 61, 94])
    x = [c.rows(rng, 94, 48) for _ in range(2)]
    x[0][5, 2], x[1][70, 40] = np.nan, np.inf
    c.table[0, 2] = -1
    with np.errstate(invalid="ignore"):
        ref.append(*x, c.lengths, c.table, start)
        q = c.rows(rng, 59, 96)
        for kw in (dict(), dict(causal=False), dict(window=20)):
            lengths = np.array([20, 1, 33]) if kw else c.lengths
            a, b = (f(ref, q, lengths, c.table, c.start, **kw) for f in (cacheref.attend, attendcases.attend))
            assert np.array_equal(np.isnan(a[0]), np.isnan(b[0])) and np.isnan(a[0]).any() and not np.isnan(a[0]).all()
            good = ~np.isnan(a[0])
            assert np.allclose(a[0][good], b[0][good], rtol=0, atol=1e-12) and np.allclose(a[1][good], b[1][good], rtol=1e-6)
