"""Refusals of the norm and cache calls that need no GPU, and the references of their tests against closed forms."""
import ctypes as C

import numpy as np
import pytest

from tests import cacheref, lbtest


@pytest.fixture(scope="module")
def lbm():
    return lbtest.ensure_built()


@pytest.fixture(scope="module")
def lib(lbm):
    return lbm.load_library()


M = 1 << 24


def _norm(lib, **kw):
    a = dict(kind=0, y=1 * M, y_type=0, ldy=64, post=0, pw=None, pb=None, gate=None, ldg=0, r=2 * M, ldr=64, scale=1.0,
             r_type=1, w=None, b=None, eps=1e-5, out=3 * M, ldo=64, x=4 * M, ldx=64, rows=4, width=64)
    a.update(kw)
    return lib.lb_norm(*a.values(), None)


@pytest.mark.parametrize("bad", [dict(kind=2), dict(kind=-1), dict(y_type=2), dict(r_type=-1), dict(rows=-1),
                                 dict(rows=(1 << 30) + 1), dict(width=0), dict(width=32769, ldy=40000, ldr=40000, ldo=40000, ldx=40000),
                                 dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=None, r=None),
                                 dict(out=None, x=None), dict(y=None, post=1), dict(y=None, gate=5 * M), dict(pw=5 * M),
                                 dict(pb=5 * M), dict(x=None, w=5 * M), dict(x=None, b=5 * M), dict(ldy=63), dict(ldr=63),
                                 dict(ldo=63), dict(ldx=63), dict(gate=5 * M, ldg=63), dict(ldy=(1 << 31) + 1),
                                 dict(y=1 * M + 1), dict(r=2 * M + 2), dict(out=3 * M + 2), dict(x=4 * M + 1), dict(w=5 * M + 1),
                                 dict(x=3 * M), dict(x=3 * M + 64), dict(out=2 * M + 4), dict(out=2 * M, ldo=128),
                                 dict(x=1 * M + 2), dict(x=1 * M, ldx=128), dict(out=1 * M), dict(gate=3 * M, ldg=0),
                                 dict(gate=4 * M, ldg=64), dict(w=4 * M), dict(post=1, pw=3 * M)])
def test_norm_refusals(lbm, lib, bad):
    assert _norm(lib, **bad) == lbm.LB_EINVAL
    assert lib.lb_last_error().startswith(b"lb_norm")


def test_norm_without_rows(lbm, lib):
    assert _norm(lib, rows=0, y=None, r=None, out=None, x=None) == lbm.LB_OK


def test_cache_refusals_without_a_cache(lbm, lib):
    out = C.c_void_p()
    good = (4, 16, 2, 64)
    for bad in ((0, 16, 2, 64), (-1, 16, 2, 64), (1 << 31, 16, 1, 64), (1 << 30, 256, 8, 64), (4, 8, 2, 64), (4, 24, 2, 64),
                (4, 512, 2, 64), (4, 16, 0, 64), (4, 16, 1025, 64), (4, 16, 2, 0), (4, 16, 2, 4), (4, 16, 2, 65),
                (4, 16, 2, 264)):
        assert lib.lb_cache_create(*bad, C.byref(out)) == lbm.LB_EINVAL, bad
        assert lib.lb_last_error().startswith(b"lb_cache_create")
    assert lib.lb_cache_create(*good, None) == lbm.LB_EINVAL
    assert out.value is None
    seq = (None, 16, 16, 4, 4, 1, 1)
    assert lib.lb_cache_append(None, 16, 128, 16, 128, None, 0, None, 0, 0, None, 0, 0, 0, *seq, None) == lbm.LB_EINVAL
    assert lib.lb_cache_read(None, 16, 128, 16, 128, *seq, None) == lbm.LB_EINVAL
    assert lib.lb_cache_attend(None, 16, 128, 2, 16, 128, *seq, 0, 1.0, 1, 0, None) == lbm.LB_EINVAL
    assert lib.lb_cache_reserve(None, 1, 1, 1, 1) == lbm.LB_EINVAL
    assert lib.lb_cache_shape(None, None, None, None, None, None) == lbm.LB_EINVAL
    assert lib.lb_cache_destroy(None) == lbm.LB_OK


def test_norm_reference():
    r = np.array([[3.0, 4.0, 0.0, 0.0]])
    (u, _), (x, tx) = cacheref.norm("rms", r=r, eps=0.0)
    assert np.allclose(u, r) and np.allclose(x, r / 2.5) and (tx < 1e-4).all()
    (u, _), (x, _) = cacheref.norm("layer", y=r, r=r, scale=2.0, gate=np.full((1, 4), 0.5), weight=np.ones(4), bias=np.full(4, 7.0),
                                   eps=0.0)
    assert np.allclose(u, 2.5 * r) and np.allclose(x.mean(), 7.0) and np.allclose(x.std(), 1.0)
    (u, _), _ = cacheref.norm("rms", y=r, post=True, post_weight=np.full(4, 2.0), eps=0.0)
    assert np.allclose(u, r * 0.8)


def test_cache_reference():
    rng = np.random.default_rng(0)
    c = cacheref.Case(rng, [20, 3], [20, 3], 16, 1, 1, 8)
    x = c.rows(rng, 23, 8)
    whole, grown = (cacheref.Cache(c.pages, 16, 1, 8) for _ in range(2))
    whole.append(x, x, c.lengths, c.table, c.start)
    for i in range(20):  # token by token: the same scales, numbers within their bound
        grown.append(x[[i]], x[[i]], c.lengths[:1] - 19 + i, c.table[:1])
    grown.append(x[20:], x[20:], c.lengths[1:], c.table[1:], np.array([0, 3]))
    assert np.array_equal(whole.scale["k"], grown.scale["k"])
    for cache in (whole, grown):
        for b in range(2):
            n = c.lengths[b]
            off = np.abs(cache.tokens("k", c.lengths, c.table, b, 0, n) - cache.tokens("k", c.lengths, c.table, b, 0, n, "true"))
            assert (off <= cache.tokens("k", c.lengths, c.table, b, 0, n, "bound") * (1 + 1e-5)).all()
    # a single key: its value; nothing to see: zeros
    one = cacheref.Cache(4, 16, 1, 8)
    v = np.full((1, 8), 127.0, np.float16)
    one.append(v, v, np.array([1]), np.array([[2]]))
    out, tol = cacheref.attend(one, np.ones((1, 8), np.float16), np.array([1]), np.array([[2]]))
    assert np.array_equal(out, v) and (tol < 0.5).all()
    out, _ = cacheref.attend(one, v, np.array([1]), np.array([[-1]]))
    assert (out == 0).all()
    # turning keeps lengths, and by position 0 everything
    rope = cacheref.rope_table(8, 6)
    y = cacheref.turn(x[:2].astype(np.float64), 5, rope, True)
    assert np.allclose((y ** 2).sum(1), (x[:2].astype(np.float64) ** 2).sum(1)) and np.allclose(y[:, 6:], x[:2, 6:])
    assert np.array_equal(cacheref.turn(x[:2].astype(np.float64), 0, rope, False), x[:2])
