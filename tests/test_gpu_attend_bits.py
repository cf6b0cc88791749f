"""Single tokens have weights of two fp16 numbers: outputs that cancel to 2^-12 of their sums (tests/attendbits.py)."""
import numpy as np
import pytest

from tests import attendbits, lbtest
from tests.lbtest import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


@pytest.mark.parametrize("dim", [8, 64, 96, 128, 256])
@pytest.mark.parametrize("sequences,pages", [(200, 1), (64, 8), (9, 60)])
def test_single_tokens(lbm, dim, sequences, pages):
    torch = lbtest.torch_dev()
    say(f"[case] attend cancelling dim={dim} pages={pages}")
    call = attendbits.Call(np.random.default_rng(dim + pages), sequences, pages, dim)
    c = call.c
    cache = lbm.Cache(c.pages, attendbits.PAGE, 1, dim)
    seq = [lbtest.to_dev(x) for x in (c.lengths, c.table)]
    cache.append(lbtest.to_dev(call.k), lbtest.to_dev(call.v), *seq, start=lbtest.to_dev(call.start))
    q = lbtest.to_dev(call.q)
    out = torch.full_like(q, float("nan"))
    want, tol = call.reference()
    cache.attend(q, out, *seq, scale=call.scale)
    off = np.abs(out.cpu().numpy().astype(np.float64) - want[:, None])
    assert (off <= tol[:, None]).all(), (off / tol[:, None]).max()
