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


def test_more_sequences_than_a_grid_has_rows(lbm):
    """Single tokens of 66000 sequences that read the same seven sequences' pages."""
    torch = lbtest.torch_dev()
    say("[case] attend 66000 sequences")
    rng = np.random.default_rng(5)
    c = cacheref.Case(rng, [1, 40, 17, 16, 0, 90, 33], [1, 1, 1, 1, 0, 1, 1], 16, 2, 4, 24)
    cache, ref = _filled(lbm, c, rng)
    q = c.rows(rng, 7, 96)
    want, tol = cacheref.attend(ref, q, c.lengths, c.table)
    which = torch.arange(66000, device="cuda") % 7
    args = [lbtest.to_dev(x)[which].contiguous() for x in (q, c.lengths, c.table)]
    out = torch.full_like(args[0], 9.0)
    cache.attend(args[0], out, *args[1:])
    assert_within(out[:7].cpu().numpy(), want, tol, "first of 66000")
    assert torch.equal(out, out[:7][which])
    # and reading as many
    k, v = (torch.full((66000, 48), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    cache.read(k, v, *args[1:])
    some = which != 4  # (the fifth has no token)
    assert torch.equal(k[some], k[:7][which][some]) and (k[~some] == 9).all() and torch.equal(v[some], v[:7][which][some])


def test_two_graphs_of_one_workspace(lbm):
    """Captured calls whose keys are cut into pieces, replayed in turn with eager ones between them."""
    torch = lbtest.torch_dev()
    say("[case] attend two graphs")
    rng = np.random.default_rng(6)
    cases = [cacheref.Case(rng, [3000, 1200], [1, 1], 32, 2, 8, 64), cacheref.Case(rng, [4500, 900], [70, 1], 32, 2, 8, 64)]
    table = np.full((4, max(c.columns for c in cases)), -1, np.int32)
    at = 0
    for i, c in enumerate(cases):
        table[2 * i: 2 * i + 2, : c.columns] = np.where(c.table >= 0, c.table + at, -1)
        at += c.pages
    cache, ref = lbm.Cache(at, 32, 2, 64), cacheref.Cache(at, 32, 2, 64)
    lengths = np.concatenate([c.lengths for c in cases])
    start = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    k, v = (cases[0].rows(rng, int(start[-1]), 128) for _ in range(2))
    cache.append(*map(lbtest.to_dev, (k, v, lengths, table)), start=lbtest.to_dev(start))
    ref.append(k, v, lengths, table, start)
    cache.reserve(71, 8, 2, 32 * table.shape[1])
    calls, wants, graphs = [], [], []
    for i, c in enumerate(cases):
        q = c.rows(rng, int(c.start[-1]), 512)
        t = np.ascontiguousarray(table[2 * i: 2 * i + 2])
        wants.append(cacheref.attend(ref, q, c.lengths, t, c.start))
        out = torch.empty(q.shape, dtype=torch.float16, device="cuda")
        calls.append((lbtest.to_dev(q), out, lbtest.to_dev(c.lengths), lbtest.to_dev(t), lbtest.to_dev(c.start)))
        cache.attend(*calls[i])
    torch.cuda.synchronize()
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            cache.attend(*call)
    for i in (0, 1, 1, 0, 0, 1):
        for call in calls:
            call[1].fill_(float("nan"))
        graphs[i].replay()
        graphs[1 - i].replay()
        for j in range(2):
            assert_within(calls[j][1].cpu().numpy(), *wants[j], f"graph {j}")
        cache.attend(*calls[i])
        assert_within(calls[i][1].cpu().numpy(), *wants[i], f"eager {i}")


def test_strides_past_32_bits(lbm):
    """Rows 2^30 + 8 numbers apart: appending (q in place), attention, reading and a norm."""
    torch = lbtest.torch_dev()
    say("[case] strides past 2^31 numbers")
    ld, dim, heads = 2 ** 30 + 8, 64, 4
    buf = torch.zeros(2 * ld + 4096, dtype=torch.float16, device="cuda")
    at = lambda first, width: buf.as_strided((3, width), (ld, 1), first)  # noqa: E731
    q, k, v, out, back = at(0, heads * dim), at(256, 64), at(320, 64), at(384, heads * dim), at(640, 64)
    torch.manual_seed(1)
    for t in (q, k, v):
        t.copy_(torch.randn(t.shape, device="cuda").half())
    rope = lbtest.to_dev(cacheref.rope_table(32, dim))
    lengths, table = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([1, 1, 1], [[0, 5], [2, 4], [3, 1]]))
    near = [t.clone().contiguous() for t in (q, k, v)]
    caches = [lbm.Cache(6, 16, 1, dim) for _ in range(2)]
    for cache, (a, b, c) in zip(caches, ((q, k, v), near)):
        cache.append(b, c, lengths, table, q=a, q_out=a, rope=rope)
    got = [torch.empty((3, w), dtype=torch.float16, device="cuda") for w in (heads * dim, 64, 64, 64)]
    caches[1].attend(near[0], got[0], lengths, table)
    caches[1].read(got[1], got[2], lengths, table)
    lbm.lb_norm(near[1], x=got[3])
    caches[0].attend(q, out, lengths, table)
    assert torch.equal(q, near[0]) and torch.equal(out, got[0])
    caches[0].read(back, out[:, :64], lengths, table)
    assert torch.equal(back, got[1]) and torch.equal(out[:, :64], got[2])
    lbm.lb_norm(k, x=back)
    assert torch.equal(back, got[3])
    del buf
