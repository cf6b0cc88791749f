"""Numbers that do not fit the C calls' ints are refused, not cut to 32 bits."""
import pytest

from tests import lbtest


@pytest.fixture(scope="module")
def lbm():
    return lbtest.ensure_built()


@pytest.mark.parametrize("bad", [(4, 2 ** 32 + 16, 2, 64), (4, 16, 2 ** 32 + 2, 64), (4, 16, 2, 2 ** 32 + 64), (4, 16 - 2 ** 32, 2, 64)])
def test_create(lbm, bad):
    with pytest.raises(ValueError):
        lbm.lb_cache_create(*bad)


def test_reserve(lbm):
    with pytest.raises(ValueError):
        lbm.lb_cache_reserve(None, 1, 2 ** 32 + 2, 1, 1)
