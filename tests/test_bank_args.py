"""Refusals of the bank and routing calls that need no GPU: bad sizes, types, strides, alignments and overlaps are
reported before any device call."""
import ctypes as C

import numpy as np
import pytest

from tests import bankref, lbtest


@pytest.fixture(scope="module")
def lbm():
    return lbtest.ensure_built()


@pytest.fixture(scope="module")
def lib(lbm):
    return lbm.load_library()


def test_null_handles(lbm, lib):
    out = C.c_void_p()
    assert lib.lb_bank_create(None, None, 1, C.byref(out)) == lbm.LB_EINVAL
    one = (C.c_void_p * 1)(None)
    arr = C.cast(one, C.c_void_p)
    assert lib.lb_bank_create(arr, None, 1, None) == lbm.LB_EINVAL
    assert lib.lb_bank_create(arr, None, 0, C.byref(out)) == lbm.LB_EINVAL
    assert lib.lb_bank_create(arr, None, 1025, C.byref(out)) == lbm.LB_EINVAL
    assert lib.lb_bank_create(arr, None, 1, C.byref(out)) == lbm.LB_EINVAL  # NULL layer
    assert out.value is None
    assert lib.lb_bank_reserve(None, 1) == lbm.LB_EINVAL
    assert lib.lb_bank_forward(None, 0, 16, 1, 64, 1, 0, 1, 0, None, None, None, 0, None) == lbm.LB_EINVAL
    assert lib.lb_bank_grouped(None, 16, 1, 1, None, 64, 1, 128, 1, 0, 0, None, None, None, 0, None) == lbm.LB_EINVAL
    assert lib.lb_bank_shape(None, None, None, None, None, None) == lbm.LB_EINVAL
    assert lib.lb_bank_destroy(None) == lbm.LB_OK
    with pytest.raises(ValueError):
        lbm.Bank([])


def _route(lib, **kw):
    a = dict(logits=1 << 20, type=1, ld=8, tokens=4, experts=8, k=2, renorm=1, ids=2 << 20, weights=3 << 20,
             offsets=4 << 20, token=5 << 20, row=6 << 20, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.lb_route(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(type=2), dict(ld=7), dict(tokens=-1), dict(tokens=1 << 30), dict(experts=0),
                                 dict(experts=1025, ld=2000), dict(k=0), dict(k=9), dict(k=65, experts=100, ld=100),
                                 dict(logits=None), dict(ids=None), dict(weights=None), dict(offsets=None),
                                 dict(token=None), dict(row=None), dict(logits=(1 << 20) + 2), dict(row=(6 << 20) + 1),
                                 dict(tokens=65), dict(tokens=65, ws=7 << 20, ws_bytes=63),
                                 dict(tokens=65, ws=None, ws_bytes=64), dict(ld=(1 << 31) + 1), dict(ids=3 << 20),
                                 dict(row=(4 << 20) + 4), dict(logits=(5 << 20) + 16),
                                 dict(tokens=65, ws=6 << 20, ws_bytes=1 << 12)])
def test_route_refusals(lbm, lib, bad):
    assert _route(lib, **bad) == lbm.LB_EINVAL
    assert lib.lb_last_error().startswith(b"lb_route")


def test_route_workspace_sizes(lbm):
    assert lbm.lb_route_ws_bytes(0, 8, 2) == 0
    assert lbm.lb_route_ws_bytes(32, 8, 2) == 0
    assert lbm.lb_route_ws_bytes(33, 8, 2) == 3 * 8 * 4
    assert lbm.lb_route_ws_bytes(4097, 8, 2) == 256 * 8 * 4
    assert lbm.lb_route_ws_bytes(1 << 20, 1024, 64) == 256 * 1024 * 4
    sizes = [lbm.lb_route_ws_bytes(t, 8, 2) for t in range(0, 9000, 7)]
    assert sizes == sorted(sizes), "enough for some tokens is enough for fewer"
    for bad in ((-1, 8, 2), (4, 0, 1), (4, 8, 0), (4, 8, 9), (1 << 30, 8, 2)):
        with pytest.raises(lbm.LBError):
            lbm.lb_route_ws_bytes(*bad)


def _combine(lib, **kw):
    a = dict(y=1 << 24, y_rows=8, ldy=16, row=2 << 24, weights=3 << 24, tokens=4, k=2, width=16, res=None, ldr=0,
             out=4 << 24, ldo=16, type=0)
    a.update(kw)
    return lib.lb_route_combine(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(type=3), dict(k=0), dict(k=65), dict(tokens=-1), dict(tokens=1 << 30),
                                 dict(y_rows=-1), dict(width=0), dict(width=(1 << 24) + 1), dict(y=None), dict(row=None),
                                 dict(weights=None), dict(out=None), dict(ldy=15), dict(ldo=15),
                                 dict(res=5 << 24, ldr=15), dict(ldo=1 << 32), dict(y=(1 << 24) + 1),
                                 dict(out=(4 << 24) + 2, type=1), dict(row=(2 << 24) + 2), dict(out=1 << 24),
                                 dict(out=(1 << 24) + 32), dict(out=2 << 24), dict(out=3 << 24),
                                 dict(res=(4 << 24) + 2, ldr=16), dict(res=4 << 24, ldr=32)])
def test_combine_refusals(lbm, lib, bad):
    assert _combine(lib, **bad) == lbm.LB_EINVAL
    assert lib.lb_last_error().startswith(b"lb_route_combine")


def test_no_tokens_launch_nothing(lbm, lib):
    assert _combine(lib, tokens=0, y=None, row=None, weights=None, out=None) == lbm.LB_OK


def test_references():
    """The float64 references of these tests against closed forms."""
    ids, w, off, token, row = bankref.route(np.array([[0.0, 1.0, 1.0], [-np.inf, np.nan, 2.0], [-np.inf] * 3]), 2, True)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1]] and off.tolist() == [0, 0, 1, 3]
    assert token.tolist() == [0, 0, 1, -1, -1, -1] and row.tolist() == [[0, 1], [2, -1], [-1, -1]]
    assert np.allclose(w, [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]], atol=1e-15)
    _, w, *_ = bankref.route(np.zeros((1, 4)), 2, False)
    assert np.allclose(w, 0.25)
    v = np.array([-3.0, 0.0, 2.0])
    assert np.allclose(bankref.act(v, "silu"), v / (1 + np.exp(-v)))
    assert np.allclose(bankref.act(v, "gelu"), bankref.act(v, "gelu_tanh"), atol=2e-3)
    assert np.allclose(bankref.act(v, "relu"), [0, 0, 2]) and bankref.act(v, "none") is v
