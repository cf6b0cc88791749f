"""Calls that attention runs with 256-row tiles: the GPU tests make them, a CPU test holds that they are such calls."""
import math

import numpy as np

from tests import cacheref

U = cacheref.U
KINDS = 3  # key heads of different data; the others repeat them

# Tokens of the sequences and how many of them are new: whole tiles, ragged ends, chunks, few rows, none.
PROMPTS = ([2100, 1, 1900], [2037, 1, 1859])
CHUNKS = ([2100, 5, 300, 620], [300, 2, 40, 300])
LONG = ([4500, 9, 70], [460, 1, 20])  # for windows of 4096 and more

WIDE = {
    "24 wide": dict(dim=24, kv=29, group=1, page=16, sequences=PROMPTS),
    "32 wide": dict(dim=32, kv=22, group=8, page=32, sequences=CHUNKS),
    "40 wide": dict(dim=40, kv=30, group=8, page=64, sequences=LONG),
    "64 wide": dict(dim=64, kv=29, group=1, page=16, sequences=PROMPTS),
    "80 wide": dict(dim=80, kv=29, group=1, page=128, sequences=PROMPTS),
    "96 wide": dict(dim=96, kv=30, group=8, page=64, sequences=LONG),
    "104 wide": dict(dim=104, kv=22, group=8, page=32, sequences=CHUNKS),
    "128 wide": dict(dim=128, kv=29, group=1, page=64, sequences=PROMPTS),
    "128 wide, long": dict(dim=128, kv=30, group=8, page=64, sequences=LONG),
}
WINDOWS = (0, 4096, 4243)  # that these calls are made with


def wide(rng, dim, kv, group, page, sequences):
    return cacheref.Case(rng, *sequences, page, kv, kv * group, dim)


def plan_arguments(c, window=0, cus=256):
    """Of tests/native/plan_print.cpp, for a call of the case with starts."""
    return [c.kv, (c.dim + 31) // 32 * 32, cus, 1, int(c.start[-1]), len(c.lengths), c.heads // c.kv, window, c.columns * c.page]


def rows(rng, c, count, per_kind, gain=1.0):
    """fp16 numbers of `per_kind` heads for each of KINDS key heads, and the same for all key heads of the case."""
    x = (rng.standard_normal((count, KINDS, per_kind * c.dim)) * gain).astype(np.float16)
    return x.reshape(count, -1), spread(c, x)


def spread(c, x):
    return np.ascontiguousarray(x.reshape(x.shape[0], KINDS, -1)[:, np.arange(c.kv) % KINDS]).reshape(x.shape[0], -1)


def attend(cache, q, lengths, table, start, causal=True, window=0):
    """cacheref.attend's outputs and tolerances by matrix products, for more keys than its element by element sums."""
    d, kv = cache.dim, cache.kv
    heads = q.shape[1] // d
    group, scale = heads // kv, d ** -0.5
    out, tol = np.full(q.shape, np.nan), np.zeros(q.shape)
    for b in range(len(lengths)):
        n = start[b + 1] - start[b]
        cap = min(max(int(lengths[b]), 0), table.shape[1] * cache.page)
        if n == 0:
            continue
        K, V = (cache.tokens(name, lengths, table, b, 0, cap) for name in "kv")
        bad = np.isnan(K).any(2) | np.isnan(V).any(2)  # [tokens, key heads]
        K, V = np.nan_to_num(K), np.nan_to_num(V)
        Q = q[start[b]: start[b + 1]].reshape(n, heads, d).astype(np.float64)
        t, pos = np.arange(cap), (int(lengths[b]) - n + np.arange(n))[:, None]
        see = np.broadcast_to(cache.seen(lengths, table, b)[None, :], (n, cap))
        if causal:
            see = see & (t <= pos)
        if window:
            see = see & (t > pos - window)
        some = see.any(1, keepdims=True)
        for h in range(heads):
            at = slice(start[b], start[b + 1]), slice(h * d, (h + 1) * d)
            if cap == 0:
                out[at] = 0
                continue
            k, v = K[:, h // group], V[:, h // group]
            z = np.where(see, scale * (Q[:, h] @ k.T), -np.inf)
            top = np.where(some, z.max(1, keepdims=True), 0.0)
            p = np.where(see, np.exp(z - top), 0.0)
            w = p / np.where(some, p.sum(1, keepdims=True), 1)
            o = w @ v
            zabs = np.where(see, scale * (np.abs(Q[:, h]) @ np.abs(k).T), 0.0)
            terr = zabs * (d + 4) * U + (np.abs(np.where(see, z, 0.0)) + np.abs(top) + 16) * 3 * U + 4 * U
            steps = 8 * math.sqrt(cap) * U
            av = np.abs(v)
            spread_ = (w * (terr + 2.0 ** -11 + steps)) @ av + cap * 2.0 ** -37 * av.max(initial=0.0)
            e = spread_ + np.abs(o) * ((w * terr).sum(1, keepdims=True) + steps + 8 * U)
            tol[at] = e + 2.0 ** -11 * (np.abs(o) + e) + 2.0 ** -25
            o[(see & bad[:, h // group]).any(1)] = np.nan
            out[at] = o
    return out, tol
