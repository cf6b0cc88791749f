"""A call of single tokens whose outputs show the roundings of attention's weights, and its reference.

Sequence b has 16 n keys of one kind and 16 n of another, each kind a key of one number, so that its score is a single exact
product and all its weights are rounded alike; its values are 1 for the first kind and -f for the second, f the fp16 number
that is nearest to the ratio of the weights.  What is left is about 2^-12 of either sum, which a weight that is rounded to
fp16 (up to 2^-11 of it, all keys of a kind one way) changes by as much again.
"""
import numpy as np

from tests import cacheref

U = 2.0 ** -24
PAGE = 16


class Call:
    def __init__(self, rng, sequences, pages, dim):
        """`pages` pages of each kind a sequence."""
        n = self.sequences = sequences
        self.dim, self.count = dim, PAGE * pages
        lengths = [2 * self.count] * n
        self.c = cacheref.Case(rng, lengths, [1] * n, PAGE, 1, 1, dim)
        key = rng.uniform(0.5, 1.5, (n, 2)).astype(np.float16)
        self.q = np.zeros((n, dim), np.float16)
        self.q[:, 0] = rng.uniform(1, 3, n).astype(np.float16)
        self.scale = 1.0
        z = self.q[:, :1].astype(np.float64) * self._held(key)
        f = np.exp(z[:, 0] - z[:, 1]).astype(np.float16)
        self.values = np.stack([np.ones(n, np.float16), -f], 1)
        rows = np.repeat(np.arange(n), 2 * self.count), np.tile(np.repeat([0, 1], self.count), n)
        self.k = np.zeros((len(rows[0]), dim), np.float16)
        self.k[:, 0] = key[rows]
        self.v = np.repeat(self.values[rows][:, None], dim, 1)
        self.z = z
        self.start = np.arange(n + 1, dtype=np.int32) * (2 * self.count)

    @staticmethod
    def _held(x):
        """What the cache holds of numbers that are their page's largest."""
        return 127 * (x.astype(np.float32) / np.float32(127)).astype(np.float64)

    def weights(self):
        """Of a key of each kind, in the largest's units."""
        return np.exp(self.z - self.z.max(1, keepdims=True))

    def output(self, w):
        """The outputs (every dim the same) of weights times value scales w [n, 2], in float64."""
        total = self.weights().sum(1)
        return (w * np.sign(self.values.astype(np.float64)) * 127).sum(1) / total

    def products(self):
        """Weight times value scale of a key of each kind."""
        return self.weights() * np.abs(self._held(self.values)) / 127

    def reference(self):
        """The outputs, and how far weights of two fp16 numbers may be from them.

        A score is one exact product: rounded with its scale, and as the exponent's argument of up to |z| + 16, three times.
        A weight times its scale is off by that, by its own two roundings and by 2^-22 (two numbers of 11 bits).  Sums of
        equal numbers over the keys: eight times the root of their number, in U.
        """
        w = self.weights() / self.weights().sum(1, keepdims=True)
        v = np.abs(self._held(self.values))
        out = self.output(self.products())
        one = (np.abs(self.z) + np.abs(self.z.max(1, keepdims=True)) + 16) * 3 * U + 6 * U
        steps = 8 * np.sqrt(2 * self.count) * U
        e = (w * (one + 2.0 ** -22 + steps) * v).sum(1) + np.abs(out) * ((w * one).sum(1) + steps + 8 * U) + 2.0 ** -36 * v.max(1)
        return out, e + 2.0 ** -11 * (np.abs(out) + e) + 2.0 ** -25


def as_half(w, numbers):
    """w as the sum of one fp16 number or two, lifted by 2^12 over the largest as the kernels lift it."""
    lift = 2.0 ** 12 / w.max(1, keepdims=True)
    hi = (w * lift).astype(np.float16).astype(np.float64)
    lo = (w * lift - hi).astype(np.float16).astype(np.float64) if numbers == 2 else 0.0
    return (hi + lo) / lift
