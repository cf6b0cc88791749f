"""Float64 references and tolerances of the bank and routing tests."""
import math

import numpy as np

import oracle

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_erfc = np.vectorize(math.erfc, otypes=[np.float64])
#: half a step of a rounding, relative to the value; and half the smallest step there is
HALF = {np.float16: 2.0 ** -11, np.float32: 2.0 ** -24}
TINY = {np.float16: 2.0 ** -25, np.float32: 2.0 ** -150}


def act(v, name):
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "gelu":
        return 0.5 * v * _erfc(-v / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v / (1.0 + np.exp(-v))
    return v


def layer(x, paths):
    """The layer on x in float64, and how far fp32 arithmetic may be from it.

    A sum of n terms in fp32 makes n roundings of at most 2^-24 of a partial sum each; with random signs they add
    up as sqrt(n), and the partial sums of the two products are of the size R_j = |h_j| |w| (root of the sum of
    squares).  The first product has a terms, the second P s; w itself carries 22 bits.  Eight times that.
    """
    a, s = paths[0]["a"], paths[0]["s"]
    w = oracle.latent(x, paths)
    y = oracle.from_latent(w, paths)
    size = np.zeros_like(y)
    for p, path in enumerate(paths):
        wp = np.sqrt((w[:, p * s:(p + 1) * s] ** 2).sum(1))
        size += np.outer(wp ** 2, path["h"].astype(np.float64) ** 2)
    steps = math.sqrt(a) + math.sqrt(len(paths) * s) + 4
    return y, 8 * 2.0 ** -24 * steps * np.sqrt(size)


def fused(x, up, gate=None, act_name="none", bias=None, gate_bias=None, residual=None, out=np.float16):
    """Reference of one layer with its epilogue and the tolerance of each element."""
    v, tv = layer(x, up)
    if bias is not None:
        v = v + bias.astype(np.float64)
        tv = tv + 2.0 ** -24 * np.abs(v)
    if gate is not None:
        g, tg = layer(x, gate)
        if gate_bias is not None:
            g = g + gate_bias.astype(np.float64)
            tg = tg + 2.0 ** -24 * np.abs(g)
        f = act(g, act_name)
        # |act'| <= 1.13; an activation in fp32 is within eight steps of its argument's and its own size
        tf = 1.13 * tg + 16 * 2.0 ** -24 * (np.abs(g) + np.abs(f))
        ref, tol = f * v, np.abs(f) * tv + (np.abs(v) + tv) * tf
    else:
        f = act(v, act_name)
        ref, tol = f, 1.13 * tv + (16 * 2.0 ** -24 * (np.abs(v) + np.abs(f)) if act_name != "none" else 0.0)
    tol = tol + 2.0 ** -23 * np.abs(ref)
    if residual is not None:
        ref = ref + residual.astype(np.float64)
        tol = tol + 2.0 ** -24 * np.abs(ref)
    return ref, tol + HALF[out] * (np.abs(ref) + tol) + TINY[out]


def assert_within(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    over = np.abs(got - ref) / tol
    assert (over <= 1.0).all(), f"{what}: {over.max():.2f} times its tolerance at {np.unravel_index(over.argmax(), over.shape)}"


def route(logits, k, renormalise):
    """The routing in float64 by repeated search, as plain loops over the tokens."""
    z = np.asarray(logits).astype(np.float64)
    z = np.where(np.isnan(z), -np.inf, z)
    t, e = z.shape
    ids = np.full((t, k), -1, np.int32)
    weights = np.zeros((t, k))
    for i in range(t):
        left = [(-z[i, j], j) for j in range(e) if z[i, j] > -np.inf]
        left.sort()
        if not left:
            continue
        top = -left[0][0]
        p = {j: 1.0 if -v == top else math.exp(-v - top) for v, j in left}
        chosen = [j for _, j in left[:k]]
        den = sum(p[j] for j in chosen) if renormalise else sum(p.values())
        for n, j in enumerate(chosen):
            ids[i, n], weights[i, n] = j, p[j] / den
    token = np.full(t * k, -1, np.int32)
    row = np.full((t, k), -1, np.int32)
    offsets = [0]
    for j in range(e):
        at = offsets[-1]
        for i, n in zip(*np.nonzero(ids == j)):
            token[at], row[i, n] = i, at
            at += 1
        offsets.append(at)
    return ids, weights, np.asarray(offsets, np.int32), token, row
