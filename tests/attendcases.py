"""Calls that attention runs with 256-row tiles: the GPU tests make them, a CPU test holds that they are such calls."""
import numpy as np

from tests import cacheref

KINDS = 3  # key heads of different data; the others repeat them

# Sequences of all sizes about a tile's, single tokens and none, in one call.
LENGTHS = [300, 1, 257, 64, 33, 700, 2, 0, 129, 90, 40, 17, 256, 255, 31, 400]
NEW = [300, 1, 257, 64, 33, 100, 2, 0, 129, 50, 33, 16, 256, 1, 31, 260]

WIDE = {
    "24 wide": dict(dim=24, kv=33, group=1, page=16),
    "32 wide": dict(dim=32, kv=9, group=8, page=32),
    "40 wide": dict(dim=40, kv=33, group=1, page=64),
    "64 wide": dict(dim=64, kv=20, group=2, page=16),
    "80 wide": dict(dim=80, kv=30, group=1, page=128),
    "96 wide": dict(dim=96, kv=33, group=1, page=16),
    "104 wide": dict(dim=104, kv=27, group=1, page=32),
    "128 wide": dict(dim=128, kv=33, group=1, page=64),
}


def wide(rng, dim, kv, group, page):
    return cacheref.Case(rng, LENGTHS, NEW, page, kv, kv * group, dim)


def plan_arguments(c, window=0, cus=256):
    """Of tests/native/plan_print.cpp, for a call of the case with starts."""
    return [c.kv, (c.dim + 31) // 32 * 32, cus, 1, int(c.start[-1]), len(c.lengths), c.heads // c.kv, window, c.columns * c.page]


def rows(rng, c, count, per_kind, gain=1.0):
    """fp16 numbers of `per_kind` heads for each of KINDS key heads, and the same for all key heads of the case."""
    x = (rng.standard_normal((count, KINDS, per_kind * c.dim)) * gain).astype(np.float16)
    return x.reshape(count, -1), spread(c, x)


def spread(c, x):
    return np.ascontiguousarray(x.reshape(x.shape[0], KINDS, -1)[:, np.arange(c.kv) % KINDS]).reshape(x.shape[0], -1)
