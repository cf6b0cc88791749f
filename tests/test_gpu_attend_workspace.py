"""The workspace of attention's calls as lengths grow without a reservation."""
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


def test_growing_bounds_keep_little_memory(lbm):
    """Chunks of 16 tokens of 32 heads on one, the bound on their lengths growing to 131072: the largest workspace is 43 MB
    for 128 wide heads, and the outgrown ones are less than twice the bound of 85 MB."""
    torch = lbtest.torch_dev()
    say("[case] attend growing max_length")
    rng = np.random.default_rng(1)
    dim, page, rows, heads, length = 128, 64, 16, 32, 300
    c = cacheref.Case(rng, [length], [rows], page, 1, heads, dim)
    table = np.full((1, 131072 // page), -1, np.int32)
    table[0, : c.columns] = c.table[0]
    cache, ref = lbm.Cache(c.pages, page, 1, dim), cacheref.Cache(c.pages, page, 1, dim)
    k, v = c.rows(rng, length, dim), c.rows(rng, length, dim)
    start = np.array([0, length], np.int32)
    cache.append(*map(lbtest.to_dev, (k, v, c.lengths, table)), start=lbtest.to_dev(start))
    ref.append(k, v, c.lengths, table, start)
    q = c.rows(rng, rows, heads * dim)
    args = [lbtest.to_dev(q), torch.empty((rows, heads * dim), dtype=torch.float16, device="cuda")]
    args += [lbtest.to_dev(x) for x in (c.lengths, table, c.start)]
    want, tol = cacheref.attend(ref, q, c.lengths, table, c.start)
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    for most in range(320, 131073, 1024):
        args[1].fill_(float("nan"))
        cache.attend(*args, max_length=most)
        if most % 16384 == 320:
            assert_within(args[1].cpu().numpy(), want, tol, f"max_length={most}")
    torch.cuda.synchronize()
    assert before - torch.cuda.mem_get_info()[0] < 3 * 86e6
