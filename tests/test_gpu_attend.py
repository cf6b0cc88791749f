"""Attention over the paged 8-bit cache, element by element (tolerances: tests/cacheref.py).

Nothing is rotated while the cache is filled, so its numbers and scales are the reference's bit for bit."""
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


def _dev(v):
    return None if v is None else lbtest.to_dev(v)


def _filled(lbm, c, rng, gain=None):
    cache, ref = lbm.Cache(c.pages, c.page, c.kv, c.dim), cacheref.Cache(c.pages, c.page, c.kv, c.dim)
    rows = int(c.lengths.sum())
    start = np.concatenate([[0], np.cumsum(c.lengths)]).astype(np.int32)
    if rows:
        k, v = c.rows(rng, rows, c.kv * c.dim, gain), c.rows(rng, rows, c.kv * c.dim, gain)
        cache.append(_dev(k), _dev(v), _dev(c.lengths), _dev(c.table), start=_dev(start))
        ref.append(k, v, c.lengths, c.table, start)
    return cache, ref


def _run(lbm, cache, ref, c, rng, what, start=True, lengths=None, table=None, qgain=1.0, q=None, **kw):
    torch = lbtest.torch_dev()
    rows = int(c.start[-1]) if start else len(c.lengths)
    q = (c.rows(rng, rows, c.heads * c.dim) * np.float16(qgain)) if q is None else q
    out = torch.full(q.shape, float("nan"), dtype=torch.float16, device="cuda")
    lengths = c.lengths if lengths is None else lengths
    table = c.table if table is None else table
    cache.attend(_dev(q), out, _dev(lengths), _dev(table), start=_dev(c.start) if start else None, **kw)
    torch.cuda.synchronize()
    most = kw.pop("max_length", 0) or 0
    want, tol = cacheref.attend(ref, q, lengths, table, c.start if start else None, most=most, **kw)
    assert_within(out.cpu().numpy(), want, tol, what)
    return q, out


@pytest.mark.parametrize("dim", [8, 24, 32, 64, 72, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 4), (3, 8), (1, 17), (2, 16)])
def test_single_tokens(lbm, dim, kv, group):
    say(f"[case] attend single dim={dim} kv={kv} group={group}")
    rng = np.random.default_rng(dim * 100 + group)
    for page in (16, 64):
        lengths = [1, 2, 15, 16, 17, 31, 33, 64, 100, 0, 257, 300]
        c = cacheref.Case(rng, lengths, [min(1, n) for n in lengths], page, kv, kv * group, dim)
        cache, ref = _filled(lbm, c, rng)
        _run(lbm, cache, ref, c, rng, f"dim={dim} page={page}", start=False)


@pytest.mark.parametrize("dim", [32, 64, 80, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("kv,group", [(1, 1), (2, 3), (1, 8), (1, 20)])
def test_chunks_and_prompts(lbm, dim, kv, group):
    """Sequences of every size class in one call: single tokens, a few, chunks, whole prompts, none."""
    say(f"[case] attend chunks dim={dim} kv={kv} group={group}")
    rng = np.random.default_rng(dim * 100 + group)
    lengths = [1, 40, 65, 200, 0, 150, 33, 130, 64, 7]
    new = [1, 1, 65, 3, 0, 50, 33, 129, 64, 0]
    for page in (16, 128):
        c = cacheref.Case(rng, lengths, new, page, kv, kv * group, dim)
        cache, ref = _filled(lbm, c, rng)
        _run(lbm, cache, ref, c, rng, f"dim={dim} page={page} causal")
        _run(lbm, cache, ref, c, rng, f"dim={dim} page={page} all", causal=False)
        _run(lbm, cache, ref, c, rng, f"dim={dim} page={page} window", window=37)


@pytest.mark.parametrize("rows", [1, 2, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_one_sequence(lbm, rows):
    """Row counts around every tile, with and without earlier tokens."""
    say(f"[case] attend one sequence rows={rows}")
    rng = np.random.default_rng(rows)
    for dim, heads, before in ((64, 1, 0), (64, 2, 61), (128, 1, 700), (192, 1, 130)):
        c = cacheref.Case(rng, [rows + before], [rows], 32, 1, heads, dim)
        cache, ref = _filled(lbm, c, rng)
        _run(lbm, cache, ref, c, rng, f"rows={rows} dim={dim} before={before}")
        _run(lbm, cache, ref, c, rng, f"rows={rows} dim={dim} before={before} window 1", window=1)


def test_widest_windows(lbm):
    """Windows past every position, with rows before position 0 in the same tile."""
    say("[case] attend widest windows")
    rng = np.random.default_rng(17)
    for new in (20, 90):
        c = cacheref.Case(rng, [100, 95], [new, new], 16, 1, 1, 64)
        cache, ref = _filled(lbm, c, rng)
        for window in (2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1):
            for lengths in (c.lengths, np.array([new - 7, 2], np.int32)):
                _run(lbm, cache, ref, c, rng, f"new={new} window={window}", lengths=lengths, window=window)


def test_scale_out_of_range(lbm):
    torch = lbtest.torch_dev()
    cache = lbm.Cache(1, 16, 1, 8)
    q, out = torch.zeros((1, 8), dtype=torch.float16, device="cuda"), torch.ones((1, 8), dtype=torch.float16, device="cuda")
    lengths, table = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    for scale in (-1.0, 1.1e6, float("inf"), float("nan")):
        with pytest.raises(lbm.LBError):
            cache.attend(q, out, lengths, table, scale=scale)
    assert (out == 1).all()


@pytest.mark.parametrize("length", [255, 256, 257, 512, 1023, 1025, 2048, 5000])
def test_split_keys(lbm, length):
    """Keys split over workgroups and joined, for single tokens and for chunks, also through a window."""
    say(f"[case] attend split length={length}")
    rng = np.random.default_rng(length)
    c = cacheref.Case(rng, [length, 3, length // 2], [1, 1, 1], 16, 2, 8, 64)
    cache, ref = _filled(lbm, c, rng)
    _run(lbm, cache, ref, c, rng, "single", start=False)
    _run(lbm, cache, ref, c, rng, "single, bound", start=False, max_length=length)
    _run(lbm, cache, ref, c, rng, "single, window", start=False, window=max(1, length - 100))
    c = cacheref.Case(rng, [length, 30, length // 2], [90, 1, 70], 32, 1, 2, 128)
    cache, ref = _filled(lbm, c, rng)
    _run(lbm, cache, ref, c, rng, "chunk")
    _run(lbm, cache, ref, c, rng, "chunk, window", window=300)
    _run(lbm, cache, ref, c, rng, "chunk, all", causal=False)


def test_long_sequence(lbm):
    """Long enough that a wave takes its keys in several batches, and for offsets far into a page table."""
    say("[case] attend 40000 keys")
    rng = np.random.default_rng(2)
    c = cacheref.Case(rng, [40000], [1], 16, 1, 3, 32)
    cache, ref = _filled(lbm, c, rng)
    _run(lbm, cache, ref, c, rng, "long", start=False)
    c.heads = 300
    _run(lbm, cache, ref, c, rng, "long, many heads", start=False)


def test_bound_on_lengths(lbm):
    """max_length below a length: the tokens past it are not seen."""
    say("[case] attend max_length")
    rng = np.random.default_rng(3)
    c = cacheref.Case(rng, [100, 50], [1, 1], 16, 1, 2, 64)
    cache, ref = _filled(lbm, c, rng)
    _run(lbm, cache, ref, c, rng, "bound 70", start=False, max_length=70)
    c = cacheref.Case(rng, [100, 50], [40, 40], 16, 1, 2, 64)
    cache, ref = _filled(lbm, c, rng)
    _run(lbm, cache, ref, c, rng, "bound 70, chunks", max_length=70)


@pytest.mark.parametrize("scale", [0.0, 0.01, 1.0, 8.0])
def test_scales_of_scores(lbm, scale):
    """From uniform weights to a single key that takes all."""
    say(f"[case] attend scale={scale}")
    rng = np.random.default_rng(4)
    for new in ([1, 1], [70, 60]):
        c = cacheref.Case(rng, [300, 90], new, 32, 2, 4, 64)
        cache, ref = _filled(lbm, c, rng)
        _run(lbm, cache, ref, c, rng, f"scale={scale}", scale=scale)


def test_scores_that_rise_and_fall(lbm):
    """Keys in order of their scores, up and down, far over the range of exp: the running reference follows."""
    say("[case] attend rising scores")
    rng = np.random.default_rng(5)
    for new in (1, 100):
        c = cacheref.Case(rng, [600, 600], [new, new], 16, 1, 1, 64)
        cache, ref = lbm.Cache(c.pages, 16, 1, 64), cacheref.Cache(c.pages, 16, 1, 64)
        k = np.ones((1200, 64), np.float16) * np.concatenate([np.linspace(-40, 40, 600), np.linspace(40, -40, 600)])[:, None].astype(np.float16)
        v = c.rows(rng, 1200, 64)
        start = np.array([0, 600, 1200], np.int32)
        cache.append(_dev(k), _dev(v), _dev(c.lengths), _dev(c.table), start=_dev(start))
        ref.append(k, v, c.lengths, c.table, start)
        _run(lbm, cache, ref, c, rng, "rising", q=np.ones((2 * new, 64), np.float16), scale=0.25)


def test_scales_of_values(lbm):
    """Pages whose values differ by seven orders of magnitude, the large ones seen or not."""
    say("[case] attend value scales")
    rng = np.random.default_rng(6)
    for new in (1, 48):
        c = cacheref.Case(rng, [160, 160], [new, new], 16, 1, 2, 64)
        cache, ref = lbm.Cache(c.pages, 16, 1, 64), cacheref.Cache(c.pages, 16, 1, 64)
        k, v = c.rows(rng, 320, 64), rng.standard_normal((320, 64))
        size = 10.0 ** rng.uniform(-3, 4, 20)
        v = (v * np.repeat(size, 16)[:, None]).clip(-65504, 65504).astype(np.float16)
        start = np.array([0, 160, 320], np.int32)
        cache.append(_dev(k), _dev(v), _dev(c.lengths), _dev(c.table), start=_dev(start))
        ref.append(k, v, c.lengths, c.table, start)
        _run(lbm, cache, ref, c, rng, "values")
        _run(lbm, cache, ref, c, rng, "values, window", window=20)


def test_what_is_not_seen_does_not_matter(lbm):
    """NaN pages behind the causal border, outside the window, past the length: no trace of them.  Seen, they are NaN."""
    torch = lbtest.torch_dev()
    say("[case] attend unseen NaN")
    rng = np.random.default_rng(7)
    for new in (20, 80):
        c = cacheref.Case(rng, [200, 150], [new, new], 16, 2, 4, 64)
        cache, ref = lbm.Cache(c.pages, 16, 2, 64), cacheref.Cache(c.pages, 16, 2, 64)
        k, v = c.rows(rng, 350, 128), c.rows(rng, 350, 128)
        k[3, 3] = np.nan      # first page of the first sequence, head 0
        v[5, 100] = np.inf    # the same page, head 1
        v[200 + 149, 7] = np.nan  # the last page of the second sequence, head 0: seen by its last rows only
        start = np.array([0, 200, 350], np.int32)
        with np.errstate(invalid="ignore"):
            cache.append(_dev(k), _dev(v), _dev(c.lengths), _dev(c.table), start=_dev(start))
            ref.append(k, v, c.lengths, c.table, start)
            _, out = _run(lbm, cache, ref, c, rng, "window", window=60)
            assert not out[:new].isnan().any() and out[new:].isnan().any() and not out[new:, 128:].isnan().any()
            if new == 80:  # rows before the last page see nothing of it
                assert not out[new: new + 74].isnan().any()
            _run(lbm, cache, ref, c, rng, "all")
            # shorter lengths: stale tokens behind them in the same page, NaN in the next
            lengths = np.array([180, 140], np.int32)
            _run(lbm, cache, ref, c, rng, "short", lengths=lengths, window=100)
    torch.cuda.synchronize()


def test_missing_pages_and_rows_without_keys(lbm):
    """Holes in the table are not attended; rows that see nothing get zeros; rows of nobody are left as they were."""
    torch = lbtest.torch_dev()
    say("[case] attend missing pages")
    rng = np.random.default_rng(8)
    for group, new in ((1, [1, 1, 1, 1]), (4, [40, 3, 1, 60])):
        c = cacheref.Case(rng, [100, 90, 70, 120], new, 16, 1, group, 64)
        cache, ref = _filled(lbm, c, rng)
        table = c.table.copy()
        table[0, [0, 3]] = -1
        table[1, 2:] = c.pages
        table[2] = 2 ** 31 - 1
        table[3, 1] = -2 ** 31
        _run(lbm, cache, ref, c, rng, "holes", table=table)
        _run(lbm, cache, ref, c, rng, "holes, window", table=table, window=16)
        lengths = np.array([0, 1, -5, 30], np.int32)  # fewer tokens than rows
        _run(lbm, cache, ref, c, rng, "short", lengths=lengths)
        _run(lbm, cache, ref, c, rng, "short, all", lengths=lengths, causal=False)
        _run(lbm, cache, ref, c, rng, "long", lengths=np.array([2 ** 31 - 1, 5000, 200, 121], np.int32), causal=False)
    c = cacheref.Case(rng, [50, 60], [30, 40], 16, 1, 1, 64)
    cache, ref = _filled(lbm, c, rng)
    q = torch.randn((80, 64), device="cuda").half()
    want = torch.empty((70, 64), dtype=torch.float16, device="cuda")
    cache.attend(q[4:74], want, _dev(c.lengths), _dev(c.table), start=_dev(c.start))
    out = torch.full((80, 64), 5.0, dtype=torch.float16, device="cuda")
    cache.attend(q, out, _dev(c.lengths), _dev(c.table), start=_dev(c.start + 4))
    assert torch.equal(out[4:74], want) and (out[:4] == 5).all() and (out[74:] == 5).all()
    for st in ([5, 2, 900], [-9, 100, 70], [80, 80, 80]):  # anything in starts stays inside the rows
        cache.attend(q, out, _dev(c.lengths), _dev(c.table), start=_dev(np.array(st, np.int32)))
        torch.cuda.synchronize()


def test_strides(lbm):
    """q and out as column blocks of wider buffers, at odd offsets."""
    torch = lbtest.torch_dev()
    say("[case] attend strides")
    rng = np.random.default_rng(9)
    for dim, new in ((64, [1, 1]), (72, [40, 2]), (128, [90, 1])):
        c = cacheref.Case(rng, [120, 33], new, 16, 2, 4, dim)
        cache, ref = _filled(lbm, c, rng)
        rows, w = sum(new), 4 * dim
        buf = torch.randn((rows, 2 * w + 3), device="cuda").half()
        q, out = buf[:, 1: 1 + w], buf[:, 2 + w: 2 + 2 * w]
        keep = buf.clone()
        cache.attend(q, out, _dev(c.lengths), _dev(c.table), start=_dev(c.start))
        want, tol = cacheref.attend(ref, q.cpu().numpy(), c.lengths, c.table, c.start)
        assert_within(out.cpu().numpy(), want, tol, f"dim={dim}")
        keep[:, 2 + w: 2 + 2 * w] = out
        assert torch.equal(buf, keep)


def test_many_sequences(lbm):
    say("[case] attend 200 sequences")
    rng = np.random.default_rng(10)
    lengths = rng.integers(0, 90, 200)
    new = np.minimum(lengths, np.where(rng.random(200) < 0.2, rng.integers(0, 80, 200), 1))
    c = cacheref.Case(rng, lengths, new, 16, 1, 4, 32)
    cache, ref = _filled(lbm, c, rng)
    _run(lbm, cache, ref, c, rng, "200 sequences")
    c = cacheref.Case(rng, lengths, np.ones(200, int), 16, 1, 4, 32)
    cache, ref = _filled(lbm, c, rng)
    _run(lbm, cache, ref, c, rng, "200 single tokens", start=False)


@pytest.mark.parametrize("sequences,heads,longest", [(70, 16, 5000), (300, 4, 4200), (9, 8, 12000)])
def test_uneven_lengths(lbm, sequences, heads, longest):
    """Single tokens of sequences of very different lengths, the long ones cut into long pieces."""
    say(f"[case] attend uneven sequences={sequences}")
    rng = np.random.default_rng(sequences)
    lengths = rng.integers(0, 60, sequences)
    lengths[[0, 5, sequences - 1]] = longest, longest // 2 + 3, longest - 17
    c = cacheref.Case(rng, lengths, np.minimum(1, lengths), 64, 4, heads, 32)
    cache, ref = _filled(lbm, c, rng)
    _run(lbm, cache, ref, c, rng, "uneven", start=False)
    _run(lbm, cache, ref, c, rng, "uneven, window", start=False, window=longest - 100)


@pytest.mark.parametrize("rows,length,kv,heads,dim", [(260, 4200, 24, 24, 32), (130, 9300, 24, 24, 40), (130, 5000, 12, 36, 160)])
def test_chunks_of_long_pieces(lbm, rows, length, kv, heads, dim):
    """Chunks with about a row tile for every third CU, whose keys are cut into long pieces: few and many of them."""
    say(f"[case] attend long pieces rows={rows} length={length}")
    rng = np.random.default_rng(rows)
    c = cacheref.Case(rng, [length, 900], [rows, 1], 64, kv, heads, dim)
    cache, ref = _filled(lbm, c, rng)
    _run(lbm, cache, ref, c, rng, "long pieces")
    _run(lbm, cache, ref, c, rng, "long pieces, window", window=4100)


def test_shared_pages_and_repeats(lbm):
    """Two sequences with a common prefix read the same pages; the same call gives the same bits."""
    torch = lbtest.torch_dev()
    say("[case] attend shared pages")
    rng = np.random.default_rng(11)
    c = cacheref.Case(rng, [64, 100], [1, 1], 16, 1, 4, 64)
    cache, ref = _filled(lbm, c, rng)
    table = c.table.copy()
    table[0, :3] = table[1, :3]
    q, out = _run(lbm, cache, ref, c, rng, "shared", start=False, table=table)
    again = torch.empty_like(out)
    for _ in range(3):
        cache.attend(_dev(q), again, _dev(c.lengths), _dev(table))
        assert torch.equal(out, again)


def test_capture_needs_the_workspace(lbm):
    torch = lbtest.torch_dev()
    say("[case] attend capture without workspace")
    rng = np.random.default_rng(12)
    c = cacheref.Case(rng, [3000], [1], 64, 1, 2, 64)
    cache, ref = _filled(lbm, c, rng)
    q = torch.randn((1, 128), device="cuda").half()
    out = torch.empty_like(q)
    args = (q, out, _dev(c.lengths), _dev(c.table))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(lbm.LBError) as ei:
            cache.attend(*args)
        out.zero_()
    assert ei.value.status == lbm.LB_ENOTREADY
    cache.reserve(1, 2, 1, 3000)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend(*args)
    g.replay()
    torch.cuda.synchronize()
    want, tol = cacheref.attend(ref, q.cpu().numpy(), c.lengths, c.table)
    assert_within(out.cpu().numpy(), want, tol, "captured")
    # the workspace grows after a capture: the graph keeps its own
    old = out.clone()
    cache.reserve(5000, 2, 4, 100000)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, old)


def test_decoding_in_a_graph(lbm):
    """Append and attend captured once, replayed for every token: lengths and pages are read on the device."""
    torch = lbtest.torch_dev()
    say("[case] decode in a graph")
    rng = np.random.default_rng(13)
    n, kv, heads, dim, page, steps = 3, 2, 4, 64, 16, 40
    columns = 4
    cache, ref = lbm.Cache(n * columns, page, kv, dim), cacheref.Cache(n * columns, page, kv, dim)
    table = rng.permutation(n * columns).reshape(n, columns).astype(np.int32)
    tdev, lengths = _dev(table), torch.zeros(n, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros((n, kv * dim), dtype=torch.float16, device="cuda") for _ in range(2))
    q, qo, out = (torch.zeros((n, heads * dim), dtype=torch.float16, device="cuda") for _ in range(3))
    cache.reserve(n, heads, n, columns * page)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.append(k, v, lengths, tdev, q=q, q_out=qo)
        cache.attend(qo, out, lengths, tdev)
    for i in range(steps):
        kh, vh = (rng.standard_normal((n, kv * dim)).astype(np.float16) for _ in range(2))
        qh = rng.standard_normal((n, heads * dim)).astype(np.float16)
        k.copy_(_dev(kh))
        v.copy_(_dev(vh))
        q.copy_(_dev(qh))
        lengths.fill_(i + 1)
        g.replay()
        torch.cuda.synchronize()
        now = np.full(n, i + 1, np.int32)
        ref.append(kh, vh, now, table)
        want, tol = cacheref.attend(ref, qh, now, table)
        assert_within(out.cpu().numpy(), want, tol, f"token {i}")


def test_two_caches_on_two_streams(lbm):
    torch = lbtest.torch_dev()
    say("[case] attend two streams")
    rng = np.random.default_rng(14)
    made = []
    for i in range(2):
        c = cacheref.Case(rng, [2000, 700], [1, 1], 32, 2, 8, 64)
        made.append((c, *_filled(lbm, c, rng), c.rows(rng, 2, 512), torch.cuda.Stream()))
    torch.cuda.synchronize()
    dev = [(_dev(q), torch.empty((2, 512), dtype=torch.float16, device="cuda"), _dev(c.lengths), _dev(c.table)) for c, _, _, q, _ in made]
    torch.cuda.synchronize()
    for _ in range(20):
        for (c, cache, ref, q, s), args in zip(made, dev):
            cache.attend(*args, stream=s)
    torch.cuda.synchronize()
    for (c, cache, ref, q, s), args in zip(made, dev):
        want, tol = cacheref.attend(ref, q, c.lengths, c.table)
        assert_within(args[1].cpu().numpy(), want, tol, "stream")
