"""Float64 references and tolerances of the norm and cache tests."""
import math

import numpy as np

HALF = {np.float16: 2.0 ** -11, np.float32: 2.0 ** -24}
TINY = {np.float16: 2.0 ** -25, np.float32: 2.0 ** -150}
U = 2.0 ** -24


# ------------------------------------------------------------------ norm
def _norm(v, tv, kind, w, b, eps):
    """N(v) w + b in float64, and how far fp32 arithmetic on values off by tv may be from it.

    A sum over a row makes at most 64 roundings of partial sums on its way (32 in a thread, then a tree over its
    threads), each at most U of the sum of the magnitudes; the quotient, the root and the products some more.
    """
    steps = 64 * U
    mean = v.mean(1, keepdims=True) if kind == "layer" else np.zeros((v.shape[0], 1))
    tm = tv.mean(1, keepdims=True) + steps * np.abs(v).mean(1, keepdims=True) if kind == "layer" else 0.0
    d = v - mean
    td = tv + tm + U * (np.abs(d) + tv + tm)
    var = (d * d).mean(1, keepdims=True) + eps
    # relative error of the variance: of its terms (2 |d| td + td^2) and of summing them
    rel = ((2 * np.abs(d) * td + td * td).mean(1, keepdims=True) + 2 * steps * (d * d).mean(1, keepdims=True)) / var + 4 * U
    assert (rel < 0.5).all(), "the test's input leaves nothing of the variance"
    rel = 0.5 * rel / (1 - rel) + 6 * U
    f = 1 / np.sqrt(var)
    n = d * f
    tn = f * td * (1 + rel) + np.abs(n) * rel + 2 * U * np.abs(n)
    if w is not None:
        n, tn = n * w, np.abs(w) * tn + U * np.abs(n * w)
    if b is not None:
        n, tn = n + b, tn + U * np.abs(n + b)
    return n, tn + U * tn


def norm(kind, r=None, y=None, weight=None, bias=None, post=False, post_weight=None, post_bias=None, gate=None, scale=1.0,
         eps=1e-5):
    """(r', its fp32 error), (x, its fp32 error): float64."""
    wide = lambda a: None if a is None else np.asarray(a).astype(np.float64)  # noqa: E731
    r, y, weight, bias, post_weight, post_bias, gate = map(wide, (r, y, weight, bias, post_weight, post_bias, gate))
    u = np.zeros_like(r) if y is None else y
    tu = np.zeros_like(u)
    if post:
        u, tu = _norm(u, tu, kind, post_weight, post_bias, eps)
    if gate is not None:
        u, tu = u * gate, np.abs(gate) * tu + U * np.abs(u * gate)
    if r is not None:
        s = float(np.float32(scale))
        u, tu = u + s * r, tu + U * (np.abs(u + s * r) + np.abs(s * r))
    return (u, tu), _norm(u, tu, kind, weight, bias, eps)


def rounded(ref, tol, dtype):
    return tol + HALF[dtype] * (np.abs(ref) + tol) + TINY[dtype]


# ----------------------------------------------------------------- cache
def rope_table(positions, rot, base=10000.0):
    angle = np.arange(positions)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def turn(x, pos, rope, interleaved):
    """x [heads, dim] in float64 at position pos."""
    if rope is None:
        return x
    rot = rope.shape[1]
    c, s = rope[pos, : rot // 2].astype(np.float64), rope[pos, rot // 2:].astype(np.float64)
    y = x.copy()
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[:, i] = x[:, i] * c - x[:, j] * s
    y[:, j] = x[:, i] * s + x[:, j] * c
    return y


class Cache:
    """Keys and values as the definition has them, page by page, in plain loops.

    Numbers are rint(value / scale) with the scale and the quotient in fp32, and rint(number * (scale / larger scale)) in
    fp64 where a page's scale grows: without a rotation every step is a single operation on fp16 inputs or on its
    results, so they are the library's bit for bit.  `error` bounds how far each number may be from the value that was
    appended, in steps: half for each rounding.
    """

    def __init__(self, pages, page, kv_heads, dim):
        self.page, self.kv, self.dim, self.pages = page, kv_heads, dim, pages
        shape = (pages, page, kv_heads, dim)
        self.num = {n: np.zeros(shape) for n in "kv"}
        self.true = {n: np.zeros(shape) for n in "kv"}
        self.error = {n: np.zeros((pages, page, kv_heads)) for n in "kv"}
        self.scale = {n: np.zeros((pages, kv_heads), np.float32) for n in "kv"}

    def append(self, k, v, lengths, table, start=None, rope=None, interleaved=False):
        n = len(lengths)
        start = np.arange(n + 1) if start is None else start
        for b in range(n):
            rows = start[b + 1] - start[b]
            at = {}
            for i in range(rows):
                p = lengths[b] - rows + i
                if p >= 0 and p // self.page < table.shape[1]:
                    at.setdefault(p // self.page, []).append((p, start[b] + i))
            for column, tokens in at.items():
                page = table[b, column]
                if not 0 <= page < self.pages:
                    continue
                self._page("k", page, tokens, k, rope, interleaved)
                self._page("v", page, tokens, v, None, False)

    def _page(self, name, page, tokens, x, rope, interleaved):
        val = {p: turn(x[r].reshape(self.kv, self.dim).astype(np.float64), p, rope, interleaved) for p, r in tokens}
        first = tokens[0][0] % self.page
        num, error = self.num[name][page], self.error[name][page]
        for h in range(self.kv):
            top = np.max([np.abs(v[h]).max() for v in val.values()])  # NaN stays
            with np.errstate(invalid="ignore"):
                s = np.float32(np.float32(top) / np.float32(127))
            if not np.isfinite(s):
                s = np.float32(np.nan)
            old = self.scale[name][page, h] if first else np.float32(0)
            if np.isnan(old) or not (s > old or np.isnan(s)):
                s = old
            elif first and not np.isnan(s):
                num[:first, h] = np.rint(num[:first, h] * (float(old) / float(s)))
                error[:first, h] = error[:first, h] * old / s + 0.5
            self.scale[name][page, h] = s
            for p, v in val.items():
                q = np.zeros(self.dim) if not s > 0 else np.rint((v[h].astype(np.float32) / s).astype(np.float32))
                num[p % self.page, h] = np.clip(q, -127, 127)
                self.true[name][page][p % self.page, h] = v[h]
                error[p % self.page, h] = 0.5

    def tokens(self, name, lengths, table, b, first, last, what="value"):
        """[tokens, heads, dim] of positions first .. last - 1; `what`: value, true or bound."""
        out = []
        for p in range(first, last):
            column = p // self.page
            page = table[b, column] if column < table.shape[1] else -1
            if not 0 <= page < self.pages:
                out.append(np.zeros((self.kv, self.dim)))
                continue
            s = self.scale[name][page].astype(np.float64)[:, None]
            if what == "value":
                out.append(self.num[name][page, p % self.page] * s)
            elif what == "true":
                out.append(self.true[name][page][p % self.page])
            else:
                out.append(np.broadcast_to(self.error[name][page][p % self.page][:, None] * s, (self.kv, self.dim)))
        return np.array(out).reshape(last - first, self.kv, self.dim)

    def seen(self, lengths, table, b):
        """Whether each token of sequence b has a page."""
        cap = min(max(int(lengths[b]), 0), table.shape[1] * self.page)
        return np.array([0 <= table[b, p // self.page] < self.pages for p in range(cap)], bool)


def attend(cache, q, lengths, table, start=None, scale=None, causal=True, window=0, most=0):
    """The outputs in float64, and for every element how far arithmetic in fp32 with fp16 weights may be from it.

    z = scale s_k (q . K): exact products, sums of D terms in fp32, three more roundings; the exponent's argument is up
    to |z| + 16 and rounded; so each weight is off by a factor 1 + t.  A weight times s_v is an fp16 number or two: off by
    2^-11 of itself, or, where it is below fp16's normal numbers, by 2^-25 where the largest weight times the largest s_v
    has 2^12 or more.  They are summed over the keys in fp32: with random signs such roundings add up as the root of their
    number; eight times that.
    """
    n, d, kv = len(lengths), cache.dim, cache.kv
    heads = q.shape[1] // d
    group = heads // kv
    scale = d ** -0.5 if scale is None else scale
    start = np.arange(n + 1) if start is None else start
    out = np.full(q.shape, np.nan)
    tol = np.zeros(q.shape)
    for b in range(n):
        rows = start[b + 1] - start[b]
        cap = min(max(int(lengths[b]), 0), table.shape[1] * cache.page)
        if most:
            cap = min(cap, most)
        if rows == 0:
            continue
        here = cache.seen(lengths, table, b)[:cap]
        K = cache.tokens("k", lengths, table, b, 0, cap)
        V = cache.tokens("v", lengths, table, b, 0, cap)
        Q = q[start[b]: start[b + 1]].reshape(rows, heads, d).astype(np.float64)
        t = np.arange(cap)
        pos = (lengths[b] - rows + np.arange(rows))[:, None]
        see = np.broadcast_to(here[None, :], (rows, cap))
        if causal:
            see = see & (t <= pos)
        if window:
            see = see & (t > pos - window)
        for h in range(heads):
            col = slice(h * d, (h + 1) * d)
            if cap == 0:
                out[start[b]: start[b + 1], col] = 0
                continue
            k, v = K[:, h // group], V[:, h // group]
            with np.errstate(invalid="ignore"):
                z = np.where(see, scale * (Q[:, h] @ k.T), -np.inf)
                zabs = np.where(see, scale * (np.abs(Q[:, h]) @ np.abs(k).T), 0.0)
                top = z.max(1, keepdims=True)
                top = np.where(np.isneginf(top), 0.0, top)
                p = np.where(see, np.exp(z - top), 0.0)
                total = p.sum(1, keepdims=True)
                some = see.any(1, keepdims=True)
                o = np.where(some, np.where(see[:, :, None], p[:, :, None] * v[None], 0.0).sum(1) / np.where(some, total, 1), 0.0)
            out[start[b]: start[b + 1], col] = o
            zs = np.where(see, z, 0.0)
            terr = zabs * (d + 4) * U + (np.abs(zs) + np.abs(top) + 16) * 3 * U + 4 * U
            w = p / np.where(some, total, 1)
            av = np.abs(np.nan_to_num(v))
            steps = 8 * math.sqrt(cap) * U
            spread = (w * (terr + 2.0 ** -11 + steps)) @ av + cap * 2.0 ** -37 * av.max(initial=0.0)
            e = spread + np.abs(o) * ((w * terr).sum(1, keepdims=True) + steps + 8 * U)
            tol[start[b]: start[b + 1], col] = e + 2.0 ** -11 * (np.abs(o) + e) + 2.0 ** -25
    return out, tol


def assert_within(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{what}: NaN in other places"
    assert np.isfinite(got[~np.isnan(got)]).all(), f"{what}: not finite"
    off = np.abs(np.nan_to_num(got) - np.nan_to_num(ref))
    bad = ~np.isnan(ref) & ~(off <= tol)
    if bad.any():
        at = np.unravel_index(np.where(bad, off, 0.0).argmax(), off.shape)
        raise AssertionError(f"{what}: {bad.sum()} values outside their tolerance, at {at} {got[at]} for {ref[at]} +- {tol[at]}")


# ----------------------------------------------------------- whole calls
class Case:
    """Sequences over randomly ordered pages: table, lengths and starts, with spare pages and columns."""

    def __init__(self, rng, lengths, new, page, kv, heads, dim, spare=2, extra_columns=1):
        self.lengths = np.asarray(lengths, np.int32)
        self.new = np.asarray(new)
        self.page, self.kv, self.heads, self.dim = page, kv, heads, dim
        used = [-(-n // page) for n in lengths]
        self.pages = sum(used) + spare
        order = rng.permutation(self.pages)
        self.columns = max(max(used, default=0) + extra_columns, 1)
        self.table = np.full((len(lengths), self.columns), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at: at + u]
            at += u
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.old = (self.lengths - self.new).astype(np.int32)
        self.old_start = np.concatenate([[0], np.cumsum(self.old)]).astype(np.int32)

    def rows(self, rng, count, width, gain=None):
        x = rng.standard_normal((count, width))
        return (x if gain is None else x * gain).astype(np.float16)
