"""The paged 8-bit cache: appending (with the rotation) and reading back, against plain loops (tests/cacheref.py)."""
import numpy as np
import pytest

from tests import cacheref, lbtest
from tests.lbtest import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


def _dev(v):
    return None if v is None else lbtest.to_dev(v)


def _read(lbm, cache, c, counts=None, fill=None):
    """Everything the cache holds of the case's sequences, as [rows, width] arrays and their starts."""
    torch = lbtest.torch_dev()
    counts = c.lengths if counts is None else np.asarray(counts)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(start[-1])
    k = torch.full((rows, c.kv * c.dim), float("nan") if fill is None else fill, dtype=torch.float16, device="cuda")
    v = k.clone()
    if rows:
        cache.read(k, v, _dev(c.lengths), _dev(c.table), start=_dev(start))
    torch.cuda.synchronize()
    return k.cpu().numpy(), v.cpu().numpy(), start


def _same(got, ref, name, c, start, what, exact):
    """Read values against the reference cache: its own (one rounding to fp16) where every step is exact; with a
    rotation, whose sums an fp32 machine rounds (3 roundings of at most sqrt(2) times the largest), a number next to a
    border may be one step off, and the scale 2^-22 of itself."""
    for b in range(len(c.lengths)):
        n = int(c.lengths[b])
        have = got[start[b]: start[b + 1]].astype(np.float64).reshape(-1, c.kv, c.dim)
        first = n - have.shape[0]
        want = ref.tokens(name, c.lengths, c.table, b, first, n)
        if exact:
            assert np.array_equal(have.astype(np.float16), want.astype(np.float16)), f"{what}: {name} of sequence {b}"
            continue
        true = ref.tokens(name, c.lengths, c.table, b, first, n, "true")
        bound = ref.tokens(name, c.lengths, c.table, b, first, n, "bound")
        # half a step for each rounding, its border 127 * 2^-21 of a step unsharp
        tol = bound * (1 + 2.0 ** -12) + 2.0 ** -11 * np.abs(true) * 1.01 + 2.0 ** -24
        off = np.abs(have - true) / tol
        assert (off <= 1).all(), f"{what}: {name} of sequence {b}: {off.max():.3f} times its tolerance"
        # the largest number of a page and head is 127 steps: its value, rounded once
        assert np.abs(have - want).max() <= 2 * bound.max() + 2.0 ** -11 * np.abs(want).max()


def _check(lbm, cache, ref, c, what, exact=True):
    k, v, start = _read(lbm, cache, c)
    _same(k, ref, "k", c, start, what, exact)
    _same(v, ref, "v", c, start, what, True)


def _q(lbm, c, q, got, rope, interleaved, what):
    got = got.cpu().numpy().astype(np.float64)
    for b in range(len(c.lengths)):
        for i in range(c.new[b]):
            r, p = c.start[b] + i, c.lengths[b] - c.new[b] + i
            want = cacheref.turn(q[r].reshape(-1, c.dim).astype(np.float64), p, rope, interleaved)
            size = np.abs(q[r].reshape(-1, c.dim).astype(np.float64)).max()
            tol = 4 * 2.0 ** -24 * size * 2 + 2.0 ** -11 * np.abs(want) * 1.01 + 2.0 ** -25
            assert (np.abs(got[r].reshape(-1, c.dim) - want) <= tol).all(), f"{what}: q of row {r}"


def _fill(lbm, c, rng, rope=None, interleaved=False, pieces=("old", "new"), gain=None, q=True):
    """A cache and its reference after the case's calls; checks the turned queries."""
    torch = lbtest.torch_dev()
    cache, ref = lbm.Cache(c.pages, c.page, c.kv, c.dim), cacheref.Cache(c.pages, c.page, c.kv, c.dim)
    width = c.kv * c.dim
    for piece in pieces:
        lengths, start = (c.old, c.old_start) if piece == "old" else (c.lengths, c.start)
        rows = int(start[-1])
        if rows == 0:
            continue
        k, v = c.rows(rng, rows, width, gain), c.rows(rng, rows, width, gain)
        qs = c.rows(rng, rows, c.heads * c.dim) if q and piece == "new" else None
        qo = None if qs is None else torch.full(qs.shape, float("nan"), dtype=torch.float16, device="cuda")
        cache.append(_dev(k), _dev(v), _dev(lengths), _dev(c.table), start=_dev(start), q=_dev(qs), q_out=qo, rope=_dev(rope),
                     interleaved=interleaved)
        ref.append(k, v, lengths, c.table, start, rope, interleaved)
        torch.cuda.synchronize()
        if qs is not None:
            _q(lbm, c, qs, qo, rope, interleaved, "q")
    return cache, ref


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim", [8, 24, 32, 64, 72, 80, 96, 128, 160, 192, 224, 248, 256])
def test_append_and_read(lbm, dim, page):
    say(f"[case] append dim={dim} page={page}")
    rng = np.random.default_rng(dim * 1000 + page)
    lengths = [1, 15, 16, 17, page - 1, page, page + 1, 2 * page + 5, 0, 40]
    new = [1, 14, 16, 1, page - 1, 1, 2, page + 7, 0, 40]
    c = cacheref.Case(rng, lengths, new, page, 2, 4, dim)
    cache, ref = _fill(lbm, c, rng)
    _check(lbm, cache, ref, c, f"dim={dim} page={page}")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (80, 40), (80, 20), (72, 72), (128, 128), (256, 256), (96, 2), (24, 10)])
def test_rotation(lbm, dim, rot, interleaved):
    say(f"[case] append dim={dim} rot={rot} interleaved={interleaved}")
    rng = np.random.default_rng(dim + rot)
    c = cacheref.Case(rng, [1, 70, 33, 5], [1, 40, 1, 5], 32, 3, 6, dim)
    rope = cacheref.rope_table(c.columns * c.page, rot)
    cache, ref = _fill(lbm, c, rng, rope, interleaved)
    _check(lbm, cache, ref, c, f"dim={dim} rot={rot}", exact=False)


def test_far_positions(lbm):
    """A rope table whose rows pass 2^31 bytes would be too large here; positions near the end of a long one instead."""
    torch = lbtest.torch_dev()
    say("[case] append at position 200000")
    rng = np.random.default_rng(4)
    n = 200001
    cache, ref = lbm.Cache(3, 256, 1, 64), cacheref.Cache(3, 256, 1, 64)
    table = np.full((1, n // 256 + 1), -1, np.int32)
    table[0, n // 256] = 2
    rope = cacheref.rope_table(table.shape[1] * 256, 64)
    k = rng.standard_normal((1, 64)).astype(np.float16)
    lengths = np.array([n], np.int32)
    cache.append(_dev(k), _dev(k), _dev(lengths), _dev(table), rope=_dev(rope))
    ref.append(k, k, lengths, table, rope=rope)
    c = cacheref.Case(rng, [1], [1], 256, 1, 1, 64)
    c.lengths, c.table = lengths, table
    gk, gv, start = _read(lbm, cache, c, [1])
    _same(gk, ref, "k", c, start, "far", False)
    _same(gv, ref, "v", c, start, "far", True)
    torch.cuda.synchronize()


def test_token_by_token_growing_scales(lbm):
    """One token a call (the form without starts), magnitudes rising so that scales grow often."""
    torch = lbtest.torch_dev()
    say("[case] append token by token")
    rng = np.random.default_rng(8)
    for page, dim in ((16, 64), (64, 96), (32, 40)):
        c = cacheref.Case(rng, [70, 41, 70], [1, 1, 1], page, 2, 2, dim)
        cache, ref = lbm.Cache(c.pages, page, 2, dim), cacheref.Cache(c.pages, page, 2, dim)
        table = _dev(c.table)
        for i in range(70):
            lengths = np.minimum(c.lengths, i + 1).astype(np.int32)  # the second stops: its last token is written again
            k, v = (rng.standard_normal((3, 2 * dim)) * (0.1 + i / 7) for _ in range(2))
            k, v = k.astype(np.float16), v.astype(np.float16)
            cache.append(_dev(k), _dev(v), _dev(lengths), table)
            ref.append(k, v, lengths, c.table)
        _check(lbm, cache, ref, c, f"page={page}")
        torch.cuda.synchronize()


def test_appending_twice_changes_nothing(lbm):
    torch = lbtest.torch_dev()
    say("[case] append twice")
    rng = np.random.default_rng(9)
    c = cacheref.Case(rng, [50, 3, 17], [20, 1, 2], 16, 2, 2, 64)
    cache, _ = _fill(lbm, c, rng, pieces=("old",))
    k, v = c.rows(rng, 23, 128) * np.float16(3), c.rows(rng, 23, 128)
    args = (_dev(k), _dev(v), _dev(c.lengths), _dev(c.table))
    cache.append(*args, start=_dev(c.start))
    once = _read(lbm, cache, c)
    cache.append(*args, start=_dev(c.start))
    again = _read(lbm, cache, c)
    assert np.array_equal(once[0], again[0]) and np.array_equal(once[1], again[1])
    torch.cuda.synchronize()


def test_zeros_small_large_and_not_finite(lbm):
    """Pages of zeros, of fp16's smallest and largest numbers, and with a NaN or an infinity, which stays in its page
    and head."""
    torch = lbtest.torch_dev()
    say("[case] append special values")
    rng = np.random.default_rng(10)
    c = cacheref.Case(rng, [16] * 5 + [40], [16] * 5 + [40], 16, 2, 2, 64)
    k, v = c.rows(rng, 120, 128), c.rows(rng, 120, 128)
    k[0:16] = v[0:16] = 0
    k[16:32] = np.float16(6e-8) * rng.integers(-1, 2, (16, 128))
    v[32:48] = 65504 * rng.integers(-1, 2, (16, 128))
    k[50, 3] = np.nan
    v[70, 127] = np.inf
    k[-1, 5] = -np.inf
    cache, ref = lbm.Cache(c.pages, 16, 2, 64), cacheref.Cache(c.pages, 16, 2, 64)
    cache.append(_dev(k), _dev(v), _dev(c.lengths), _dev(c.table), start=_dev(c.start))
    with np.errstate(invalid="ignore"):
        ref.append(k, v, c.lengths, c.table, c.start)
        gk, gv, start = _read(lbm, cache, c)
        for got, name in ((gk, "k"), (gv, "v")):
            for b in range(6):
                want = ref.tokens(name, c.lengths, c.table, b, 0, int(c.lengths[b])).astype(np.float16)
                have = got[start[b]: start[b + 1]].reshape(want.shape)
                assert np.array_equal(have, want, equal_nan=True), (name, b)
    assert np.isnan(gk[48:64, :64]).all() and not np.isnan(gk[48:64, 64:]).any() and not np.isnan(gk[64:80]).any()
    # a page that begins again is well again
    k2 = c.rows(rng, 120, 128)
    cache.append(_dev(k2), _dev(k2), _dev(c.lengths), _dev(c.table), start=_dev(c.start))
    gk, gv, _ = _read(lbm, cache, c)
    assert np.isfinite(gk).all() and np.isfinite(gv).all()
    torch.cuda.synchronize()


def test_rows_and_pages_that_do_not_exist(lbm):
    """Pages outside the cache, lengths past the table and below the rows, starts out of range: nothing else changes."""
    torch = lbtest.torch_dev()
    say("[case] append bad pages")
    rng = np.random.default_rng(11)
    c = cacheref.Case(rng, [64, 64, 64, 64], [64, 64, 64, 64], 16, 1, 1, 64, extra_columns=0)
    cache, ref = _fill(lbm, c, rng)
    good = _read(lbm, cache, c)
    table = c.table.copy()
    table[0] = -1
    table[1] = c.pages + 5
    table[2, 1:] = 2 ** 31 - 1
    lengths = np.array([64, 64, 80, 3], np.int32)  # the third is longer than its table, the last shorter than its rows
    start = np.array([3, 20, 40, 45, 60], np.int32)  # rows before and behind are nobody's
    x = c.rows(rng, 64, 64)
    q = c.rows(rng, 64, 64)
    qo = torch.full((64, 64), 7.0, dtype=torch.float16, device="cuda")
    cache.append(_dev(x), _dev(x), _dev(lengths), _dev(table), start=_dev(start), q=_dev(q), q_out=qo)
    # of the third, rows 40 .. 44 are positions 75 .. 79: none; of the last, rows 57 .. 59 are positions 0 .. 2
    ref.append(x, x, lengths, table, start)
    _check(lbm, cache, ref, c, "bad pages")
    k, v, _ = _read(lbm, cache, c)
    same = np.ones(256, bool)
    same[192:208] = False  # the page that begins again at row 57
    assert np.array_equal(k[same], good[0][same]) and np.array_equal(v[same], good[1][same])
    got = qo.cpu().numpy()
    turned = np.zeros(64, bool)
    turned[3:40] = turned[57:60] = True  # rows with a position in the table, whether it has a page or not
    assert np.array_equal(got[turned], q[turned]) and (got[~turned] == 7).all()
    # reading: rows without a page are zeros, rows without a position are left
    c2 = cacheref.Case(rng, [64], [64], 16, 1, 1, 64)
    c2.lengths, c2.table = np.array([5, 20], np.int32), np.array([[2 ** 30], [-7]], np.int32)
    k, v, _ = _read(lbm, cache, c2, [9, 18], fill=3.0)
    assert (k[:4] == 3).all() and (k[4:] == 0).all() and (v[:4] == 3).all() and (v[4:] == 0).all()
    # starts that fall or leave the rows, lengths below zero
    for st, ln in (([5, 2, 900, -4, 64], [64, 64, 64, 64]), ([-9, 10, 10, 70, 70], [-1, 2 ** 31 - 1, 0, 1])):
        cache.append(_dev(x), _dev(x), _dev(np.array(ln, np.int32)), _dev(c.table), start=_dev(np.array(st, np.int32)), q=_dev(q),
                     q_out=qo)
        torch.cuda.synchronize()


def test_strides_and_queries_in_place(lbm):
    """q, k and v as column blocks of one projection's rows, at odd offsets; q turned in place."""
    torch = lbtest.torch_dev()
    say("[case] append strides")
    rng = np.random.default_rng(12)
    for dim, heads, kv, inter, rot in ((64, 6, 2, False, 64), (80, 9, 3, True, 40), (80, 9, 3, False, 40), (128, 32, 8, False, 128)):
        c = cacheref.Case(rng, [21, 40, 9], [21, 1, 5], 16, kv, heads, dim)
        rope = cacheref.rope_table(c.columns * 16, rot)
        rows, kw, qw = 27, kv * dim, heads * dim
        buf = torch.randn((rows, qw + 2 * kw + 3), device="cuda").half()
        q, k, v = buf[:, 1: 1 + qw], buf[:, 1 + qw: 1 + qw + kw], buf[:, 2 + qw + kw: 2 + qw + 2 * kw]
        keep = buf.clone()
        one, two = lbm.Cache(c.pages, 16, kv, dim), lbm.Cache(c.pages, 16, kv, dim)
        seq = (_dev(c.lengths), _dev(c.table))
        qo = torch.empty((rows, qw), dtype=torch.float16, device="cuda")
        one.append(k.contiguous(), v.contiguous(), *seq, start=_dev(c.start), q=q.contiguous(), q_out=qo, rope=_dev(rope), interleaved=inter)
        two.append(k, v, *seq, start=_dev(c.start), q=q, q_out=q, rope=_dev(rope), interleaved=inter)
        torch.cuda.synchronize()
        assert torch.equal(q, qo)
        keep[:, 1: 1 + qw] = qo
        assert torch.equal(buf, keep)
        c.lengths[1] = 1  # (the second sequence's earlier tokens were never written)
        a, b = _read(lbm, one, c, [21, 0, 5]), _read(lbm, two, c, [21, 0, 5])
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_many_sequences(lbm):
    """More sequences than a wave looks at in one step, some of them empty."""
    say("[case] append 300 sequences")
    rng = np.random.default_rng(13)
    lengths = rng.integers(0, 40, 300)
    new = np.minimum(lengths, rng.integers(0, 5, 300) * rng.integers(0, 5, 300))
    c = cacheref.Case(rng, lengths, new, 16, 1, 2, 32)
    cache, ref = _fill(lbm, c, rng)
    _check(lbm, cache, ref, c, "300 sequences")


def test_addresses_past_32_bits(lbm):
    """The last page of a cache of 5 GB of keys."""
    torch = lbtest.torch_dev()
    say("[case] append past 2^32 bytes")
    rng = np.random.default_rng(14)
    pages = 40000
    cache, ref = lbm.Cache(pages, 64, 8, 256), cacheref.Cache(2, 64, 8, 256)
    table = np.array([[pages - 1, 0]], np.int32)
    lengths, start = np.array([70], np.int32), np.array([0, 70], np.int32)
    k, v = (rng.standard_normal((70, 2048)).astype(np.float16) for _ in range(2))
    cache.append(_dev(k), _dev(v), _dev(lengths), _dev(table), start=_dev(start))
    ref.append(k, v, lengths, np.array([[1, 0]]), start)
    c = cacheref.Case(rng, [70], [70], 64, 8, 8, 256)
    c.lengths, c.table = lengths, table
    gk, gv, st = _read(lbm, cache, c)
    c.table = np.array([[1, 0]])
    _same(gk, ref, "k", c, st, "far", True)
    _same(gv, ref, "v", c, st, "far", True)
    # and its keys as attention reads them
    q = torch.randn((1, 2048), device="cuda").half()
    out = torch.empty_like(q)
    cache.attend(q, out, _dev(lengths), _dev(table))
    want, tol = cacheref.attend(ref, q.cpu().numpy(), lengths, c.table)
    cacheref.assert_within(out.cpu().numpy(), want, tol, "far")
    cache.close()


def test_refusals(lbm):
    torch = lbtest.torch_dev()
    say("[case] cache refusals")
    cache = lbm.Cache(4, 16, 2, 64)
    assert lbm.lb_cache_shape(cache.handle) == (4, 16, 2, 64, torch.cuda.current_device())
    f = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    k, q, rope = f(3, 128), f(3, 256), torch.zeros((32, 64), device="cuda")
    good = dict(k=k, v=f(3, 128), lengths=i(3), table=i(3, 2))
    cache.append(**good)
    bad = [dict(k=f(3, 64)), dict(v=f(2, 128)), dict(k=k.float()), dict(k=k.cpu()), dict(lengths=i(2)), dict(lengths=i(3).long()),
           dict(table=i(2, 2)), dict(table=i(3, 2).long()), dict(start=i(3)), dict(q=q), dict(q_out=q), dict(q=q, q_out=f(3, 128)),
           dict(q=f(2, 256), q_out=f(2, 256)), dict(q=f(3, 96), q_out=f(3, 96)), dict(rope=rope.double()), dict(rope=rope[0]),
           dict(table=i(4, 3).t())]
    for kw in bad:
        with pytest.raises(ValueError):
            cache.append(**{**good, **kw})
    for kw in (dict(rope=rope[:31].contiguous()), dict(rope=torch.zeros((32, 66), device="cuda")),
               dict(rope=torch.zeros((32, 63), device="cuda")), dict(table=i(3, 0)),
               dict(q=q, q_out=q.view(-1)[:768].view(3, 256)[:, :].as_strided((3, 256), (128, 1)))):
        with pytest.raises((lbm.LBError, ValueError)):
            cache.append(**{**good, **kw})
    with pytest.raises(lbm.LBError):  # q over k
        cache.append(**{**good, "q": q[:, :128], "q_out": k})
    with pytest.raises(lbm.LBError):
        cache.read(k, k, i(3), i(3, 2))
    out = f(3, 256)
    seq = dict(lengths=i(3), table=i(3, 2))
    cache.attend(q, out, **seq)
    for kw in (dict(q=f(3, 100)), dict(out=f(2, 256)), dict(out=f(3, 128)), dict(out=out.float()), dict(start=i(3)), dict(lengths=i(4))):
        with pytest.raises(ValueError):
            cache.attend(**{"q": q, "out": out, **seq, **kw})
    for kw in (dict(q=f(3, 192), out=f(3, 192)), dict(out=q), dict(scale=-1.0), dict(scale=float("nan")), dict(window=-1),
               dict(window=4, causal=False), dict(max_length=-1)):
        with pytest.raises(lbm.LBError):
            cache.attend(**{"q": q, "out": out, **seq, **kw})
    for args in ((4, 3, 1, 9), (-1, 2, 1, 9), (1, 2, -1, 9), (1, 2, 1, -1)):
        with pytest.raises(lbm.LBError):
            cache.reserve(*args)
    e = f(0, 128)
    cache.append(e, e, i(0), i(0, 2))
    cache.attend(f(0, 256), f(0, 256), i(0), i(0, 2))
    cache.append(e, e, i(3), i(3, 2), start=i(4))
    torch.cuda.synchronize()
