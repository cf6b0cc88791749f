"""Attention at the ends of its ranges, element by element (tolerances: tests/cacheref.py)."""
import numpy as np
import pytest

from tests import cacheref, lbtest
from tests.cacheref import assert_within
from tests.lbtest import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


def _filled(lbm, c, rng, k_sign=None):
    cache, ref = lbm.Cache(c.pages, c.page, c.kv, c.dim), cacheref.Cache(c.pages, c.page, c.kv, c.dim)
    rows = int(c.lengths.sum())
    start = np.concatenate([[0], np.cumsum(c.lengths)]).astype(np.int32)
    k, v = c.rows(rng, rows, c.kv * c.dim), c.rows(rng, rows, c.kv * c.dim)
    if k_sign is not None:
        k = np.abs(k) * np.float16(k_sign) + np.float16(0.5 * k_sign)
    cache.append(*map(lbtest.to_dev, (k, v, c.lengths, c.table)), start=lbtest.to_dev(start))
    ref.append(k, v, c.lengths, c.table, start)
    return cache, ref


def _run(cache, ref, c, q, what, start=True, **kw):
    torch = lbtest.torch_dev()
    out = torch.full(q.shape, 9.0, dtype=torch.float16, device="cuda")
    starts = c.start if start else None
    cache.attend(lbtest.to_dev(q), out, *map(lbtest.to_dev, (c.lengths, c.table)), start=lbtest.to_dev(starts) if start else None, **kw)
    with np.errstate(invalid="ignore"):
        want, tol = cacheref.attend(ref, q, c.lengths, c.table, starts, **kw)
        assert_within(out.cpu().numpy(), want, tol, what)
    return want


@pytest.mark.parametrize("dim", [8, 40, 64, 128, 160, 256])
def test_queries_that_are_not_finite(lbm, dim):
    """A row whose q has an infinity or a NaN is NaN if it sees a token, also where all its scores are -inf; the rows and
    heads beside it are as they would be."""
    say(f"[case] attend infinite q dim={dim}")
    rng = np.random.default_rng(dim)
    for sign in (1, -1):
        for lengths, new, start in (([1, 2, 40, 300], [1] * 4, False), ([5, 60, 1, 30], [5, 60, 1, 0], True),
                                    ([150, 700], [150, 40], True)):
            c = cacheref.Case(rng, lengths, new, 16, 2, 4, dim)
            cache, ref = _filled(lbm, c, rng, sign)
            q = c.rows(rng, sum(new), 4 * dim)
            for r, h, x in ((0, 0, np.inf), (0, 1, -np.inf), (1, 2, np.inf), (1, 3, np.nan), (2, 0, -np.inf), (3, 1, np.inf)):
                q[r % len(q), h * dim + r * 5 % dim] = x
            want = _run(cache, ref, c, q, f"dim={dim} sign={sign} new={new}", start=start)
            assert np.isnan(want[0, :dim]).all() and not np.isnan(want[0, 2 * dim:]).any()
