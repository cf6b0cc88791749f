"""The bound on two-number weights (tests/attendbits.py) has teeth: one fp16 number a weight fails it."""
import numpy as np
import pytest

from tests import attendbits, cacheref


@pytest.mark.parametrize("pages", [1, 8])
def test_bound(pages):
    call = attendbits.Call(np.random.default_rng(pages), 200, pages, 8)
    want, tol = call.reference()
    two, one = (call.output(attendbits.as_half(call.products(), n)) for n in (2, 1))
    assert (np.abs(two - want) <= tol).all()
    assert (np.abs(one - want) > tol).mean() > 0.5


def test_reference():
    """The closed form against the plain loops."""
    call = attendbits.Call(np.random.default_rng(3), 5, 2, 8)
    c = call.c
    ref = cacheref.Cache(c.pages, attendbits.PAGE, 1, 8)
    ref.append(call.k, call.v, c.lengths, c.table, call.start)
    want, _ = cacheref.attend(ref, call.q, c.lengths, c.table, scale=call.scale)
    assert np.abs(want - call.reference()[0][:, None]).max() < 1e-12
