"""Attention in tiles of 256 rows (calls with many rows a sequence, heads up to 128 wide), element by element.

A few key heads have data of their own and are held against float64; the others repeat them and must give the same bits."""
import numpy as np
import pytest

from tests import attendcases, cacheref, lbtest
from tests.attendcases import KINDS, WIDE, WINDOWS
from tests.cacheref import assert_within
from tests.lbtest import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


def _filled(lbm, c, rng, spoil=None, k_gain=1.0):
    cache, ref = lbm.Cache(c.pages, c.page, c.kv, c.dim), cacheref.Cache(c.pages, c.page, KINDS, c.dim)
    count = int(c.lengths.sum())
    start = np.concatenate([[0], np.cumsum(c.lengths)]).astype(np.int32)
    k, v = (attendcases.rows(rng, c, count, 1, g)[0] for g in (k_gain, 1.0))
    if spoil:
        spoil(k, v, start)
    with np.errstate(invalid="ignore"):
        cache.append(*(lbtest.to_dev(x) for x in (attendcases.spread(c, k), attendcases.spread(c, v), c.lengths, c.table)),
                     start=lbtest.to_dev(start))
        ref.append(k, v, c.lengths, c.table, start)
    return cache, ref


def _run(cache, ref, c, rng, what, lengths=None, table=None, **kw):
    torch = lbtest.torch_dev()
    count, group = int(c.start[-1]), c.heads // c.kv
    lengths = c.lengths if lengths is None else lengths
    table = c.table if table is None else table
    q, full = attendcases.rows(rng, c, count, group)
    out = torch.full((count, c.heads * c.dim), float("nan"), dtype=torch.float16, device="cuda")
    cache.attend(lbtest.to_dev(full), out, lbtest.to_dev(lengths), lbtest.to_dev(table), start=lbtest.to_dev(c.start), **kw)
    torch.cuda.synchronize()
    got = out.cpu().numpy().reshape(count, c.kv, group * c.dim)
    mine = np.ascontiguousarray(got[:, :KINDS])
    assert np.array_equal(got, mine[:, np.arange(c.kv) % KINDS], equal_nan=True), f"{what}: heads of the same data differ"
    with np.errstate(invalid="ignore"):
        want, tol = attendcases.attend(ref, q, lengths, table, c.start, **kw)
        assert_within(mine.reshape(count, -1), want, tol, what)
    return mine


@pytest.mark.parametrize("name", list(WIDE))
def test_masks(lbm, name):
    say(f"[case] attend 256-row tiles, {name}")
    rng = np.random.default_rng(len(name) * 100 + WIDE[name]["dim"])
    c = attendcases.wide(rng, **WIDE[name])
    cache, ref = _filled(lbm, c, rng)
    _run(cache, ref, c, rng, name + ", causal")
    _run(cache, ref, c, rng, name + ", all", causal=False)
    if c.lengths[0] > 4096:
        for window in WINDOWS[1:]:
            _run(cache, ref, c, rng, name + f", window {window}", window=window)


@pytest.mark.parametrize("name", ["24 wide", "64 wide", "80 wide", "104 wide", "128 wide"])
def test_holes_and_short_lengths(lbm, name):
    say(f"[case] attend 256-row tiles, holes, {name}")
    rng = np.random.default_rng(WIDE[name]["dim"])
    c = attendcases.wide(rng, **WIDE[name])
    cache, ref = _filled(lbm, c, rng)
    table = c.table.copy()
    table[0, 0] = -1
    table[0, 2:5] = 2 ** 31 - 1
    table[0, 7] = c.pages
    table[2, 1::2] = -2 ** 31
    _run(cache, ref, c, rng, name + ", holes", table=table)
    _run(cache, ref, c, rng, name + ", holes, all", table=table, causal=False)
    lengths = c.lengths.copy()
    lengths[0], lengths[2] = c.new[0] - 301, 2 ** 31 - 1  # below its rows; past the table
    _run(cache, ref, c, rng, name + ", other lengths", lengths=lengths)
    lengths[0], lengths[1], lengths[2] = 1, -7, 90
    _run(cache, ref, c, rng, name + ", few tokens", lengths=lengths)
    _run(cache, ref, c, rng, name + ", few tokens, all", lengths=lengths, causal=False)


@pytest.mark.parametrize("name", ["32 wide", "64 wide", "96 wide", "128 wide"])
def test_nan_behind_masks(lbm, name):
    """NaN pages are NaN to the rows that see them and nothing to the others."""
    say(f"[case] attend 256-row tiles, NaN, {name}")
    rng = np.random.default_rng(WIDE[name]["dim"] + 1)
    c = attendcases.wide(rng, **WIDE[name])
    old, new = int(c.lengths[0] - c.new[0]), int(c.new[0])

    def spoil(k, v, start):
        k[start[0] + 3, 1] = np.nan  # an early page of key head 0
        v[start[1] - 1, c.dim + 2] = np.inf  # the first sequence's last one, of key head 1
        v[start[0] + old + new // 2, 2 * c.dim] = -np.inf  # one among its rows, of key head 2

    cache, ref = _filled(lbm, c, rng, spoil)
    for kw in (dict(), dict(causal=False), dict(window=4200)):
        some = _run(cache, ref, c, rng, f"{name} {kw}", **kw)
        seen = np.isnan(some).any(2)[:new]  # [rows, kinds]
        if kw.get("causal", True):
            assert not seen[: new // 2 - c.page, 1:].any() and seen[-1].tolist() == [c.lengths[0] <= 4200 or not kw, True, True]


@pytest.mark.parametrize("name", ["64 wide", "128 wide"])
def test_sharp_scores_and_rows_of_nobody(lbm, name):
    """Scores far over the range of exp; rows before and behind the sequences are left as they were."""
    torch = lbtest.torch_dev()
    say(f"[case] attend 256-row tiles, sharp, {name}")
    rng = np.random.default_rng(WIDE[name]["dim"] + 2)
    c = attendcases.wide(rng, **WIDE[name])
    cache, ref = _filled(lbm, c, rng, k_gain=20.0)
    _run(cache, ref, c, rng, name + ", sharp")
    count = int(c.start[-1])
    q = torch.randn((count + 9, c.heads * c.dim), device="cuda").half()
    want, out = torch.empty_like(q[4: 4 + count]), torch.full_like(q, 5.0)
    seq = [lbtest.to_dev(x) for x in (c.lengths, c.table)]
    cache.attend(q[4: 4 + count], want, *seq, start=lbtest.to_dev(c.start))
    cache.attend(q, out, *seq, start=lbtest.to_dev((c.start + 4).astype(np.int32)))
    assert torch.equal(out[4: 4 + count], want) and (out[:4] == 5).all() and (out[4 + count:] == 5).all()
    again = torch.empty_like(want)
    for _ in range(5):
        cache.attend(q[4: 4 + count], again, *seq, start=lbtest.to_dev(c.start))
        assert torch.equal(again, want)
