"""Routing where the ways through its kernels change: one workgroup against many, a wave's second set of 64 rows."""
import numpy as np
import pytest

from tests import bankref, lbtest
from tests.lbtest import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


def _check(lbm, z, k, what):
    """Whole numbers equal; weights within the roundings of exp's argument, exp, the sum and the quotient."""
    r = lbm.Route(z.shape[0], z.shape[1], k).run(lbtest.to_dev(z))
    ids, w, off, token, row = bankref.route(z, k, True)
    for got, want, name in ((r.experts, ids, "experts"), (r.offsets, off, "offsets"), (r.token, token, "token"),
                            (r.row, row, "row")):
        assert np.array_equal(got.cpu().numpy(), want), f"{what}: {name}"
    top = np.abs(np.where(np.isfinite(z), z, 0).astype(np.float64)).max(initial=0.0)
    steps = 2 * (2 * top + 2 + z.shape[1] + 2)
    assert (np.abs(r.weights.cpu().numpy() - w) <= 2.0 ** -24 * steps * w + 2.0 ** -149).all(), f"{what}: weights"


@pytest.mark.parametrize("tokens", [16, 17, 31, 32, 33, 47, 48, 49])
@pytest.mark.parametrize("experts,k", [(8, 2), (65, 64), (64, 64)])
def test_few_tokens(lbm, tokens, experts, k):
    """Up to 32 tokens one workgroup routes alone: a second token for a wave from 17 on, more than 64 rows of it
    from 1025 rows on."""
    say(f"[case] route tokens={tokens} experts={experts} k={k}")
    rng = np.random.default_rng(tokens)
    _check(lbm, rng.standard_normal((tokens, experts)).astype(np.float32), k, "no ties")
    _check(lbm, rng.integers(-2, 3, (tokens, experts)).astype(np.float16), k, "ties")
    z = rng.standard_normal((tokens, experts)).astype(np.float32)
    z[rng.random(z.shape) < 0.5] = -np.inf
    _check(lbm, z, k, "half of them masked")


@pytest.mark.parametrize("tokens,experts,k", [(6000, 64, 48), (6001, 64, 63), (5000, 300, 64), (4500, 64, 64), (5000, 1024, 60)])
def test_many_rows_in_a_block(lbm, tokens, experts, k):
    """A block of more than 1024 rows: a wave places several sets of 64, each behind the ones before it."""
    say(f"[case] route tokens={tokens} experts={experts} k={k}")
    rng = np.random.default_rng(tokens + k)
    z = rng.integers(-3, 4, (tokens, experts)).astype(np.float16)  # ties
    z[::7, :5] = -np.inf
    z[3::11] = -np.inf
    z[4::11, 2:] = np.nan
    _check(lbm, z, k, "ties")
