"""The cache's calls at the ends of their ranges."""
import numpy as np
import pytest

from tests import cacheref, lbtest
from tests.lbtest import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


@pytest.mark.parametrize("rows", [1, 15, 16, 300])
def test_rows_of_no_sequences(lbm, rows):
    """Rows and no sequences: nobody's rows, left as they were."""
    torch = lbtest.torch_dev()
    say(f"[case] no sequences, rows={rows}")
    rng = np.random.default_rng(rows)
    c = cacheref.Case(rng, [40], [40], 16, 2, 4, 64)
    cache = lbm.Cache(c.pages, 16, 2, 64)
    x = lbtest.to_dev(c.rows(rng, 40, 128))
    seq = (lbtest.to_dev(c.lengths), lbtest.to_dev(c.table))
    cache.append(x, x, *seq, start=lbtest.to_dev(c.start))
    none = dict(lengths=torch.empty(0, dtype=torch.int32, device="cuda"), table=torch.empty((0, 3), dtype=torch.int32, device="cuda"),
                start=torch.zeros(1, dtype=torch.int32, device="cuda"))
    k, q = (torch.full((rows, w), 3.0, dtype=torch.float16, device="cuda") for w in (128, 256))
    for extra in ({}, dict(q=q, q_out=torch.full_like(q, 5.0))):
        cache.append(k, k, **none, **extra)
        assert "q" not in extra or (extra["q_out"] == 5).all()
    out = [torch.full_like(t, 7.0) for t in (k, k, q)]
    cache.read(out[0], out[1], **none)
    cache.attend(q, out[2], **none)
    assert all((t == 7).all() for t in out)
    back = [torch.empty((40, 128), dtype=torch.float16, device="cuda") for _ in range(4)]
    cache.read(back[0], back[1], *seq, start=lbtest.to_dev(c.start))
    fresh = lbm.Cache(c.pages, 16, 2, 64)
    fresh.append(x, x, *seq, start=lbtest.to_dev(c.start))
    fresh.read(back[2], back[3], *seq, start=lbtest.to_dev(c.start))
    assert torch.equal(back[0], back[2]) and torch.equal(back[1], back[3])
    torch.cuda.synchronize()


def test_after_a_cache_that_does_not_fit(lbm):
    """A cache of 8.8 TB is refused, and the calls behind it are not told of that."""
    torch = lbtest.torch_dev()
    say("[case] cache that does not fit")
    r, x = torch.randn((2, 64), device="cuda"), torch.empty((2, 64), dtype=torch.float16, device="cuda")
    for _ in range(2):
        with pytest.raises(lbm.LBError) as ei:
            lbm.Cache(2 ** 31 - 1, 16, 1, 256)
        assert ei.value.status == lbm.LB_ENOMEM
        lbm.lb_norm(r, x=x)
    torch.cuda.synchronize()
    want = r / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-5)
    assert (x.float() - want).abs().max() < 1e-2  # (test_gpu_norm has its tolerances)


def test_windows_past_32_bits(lbm):
    """A window wider than any position hides nothing, whatever its lower bits; below zero there is none."""
    torch = lbtest.torch_dev()
    say("[case] windows past 32 bits")
    rng = np.random.default_rng(3)
    c = cacheref.Case(rng, [90, 40], [50, 1], 16, 1, 2, 64)
    cache = lbm.Cache(c.pages, 16, 1, 64)
    x, start = lbtest.to_dev(c.rows(rng, 130, 64)), lbtest.to_dev(np.array([0, 90, 130], np.int32))
    seq = (lbtest.to_dev(c.lengths), lbtest.to_dev(c.table))
    cache.append(x, x, *seq, start=start)
    q = lbtest.to_dev(c.rows(rng, 51, 128))
    out, want = torch.empty_like(q), torch.empty_like(q)
    cache.attend(q, want, *seq, start=lbtest.to_dev(c.start))
    for window in (2 ** 31, 2 ** 32 - 1, 2 ** 32 + 5, 2 ** 63 - 1):
        out.fill_(float("nan"))
        cache.attend(q, out, *seq, start=lbtest.to_dev(c.start), window=window)
        assert torch.equal(out, want), window
    for window in (-2 ** 31, -2 ** 32 + 5, -2 ** 63):
        with pytest.raises(lbm.LBError):
            cache.attend(q, out, *seq, start=lbtest.to_dev(c.start), window=window)
