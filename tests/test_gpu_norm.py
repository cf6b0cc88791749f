"""lb_norm against the float64 reference, element by element (tolerances: tests/cacheref.py)."""
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


def _inputs(rng, rows, width, y, r, affine, post, gate, kind):
    f = lambda *shape: rng.standard_normal(shape)  # noqa: E731
    a = {"r": None if r is None else (f(rows, width) * 3).astype(r), "y": None if y is None else (f(rows, width) + 0.5).astype(y)}
    for name in ("weight", "bias", "post_weight", "post_bias"):
        use = affine and (post or not name.startswith("post"))
        a[name] = (f(width) * 0.3 + (1 if name.endswith("weight") else 0)).astype(np.float16) if use else None
    a["gate"] = None if gate is None else f(rows if gate == "rows" else 1, width).astype(np.float16)
    return a


def _run(lbm, rng, rows, width, kind="rms", y=np.float16, r=np.float32, affine=True, post=False, gate=None, scale=1.0,
         out=None, eps=1e-5, data=None):
    torch = lbtest.torch_dev()
    a = data or _inputs(rng, rows, width, y, r, affine, post, gate, kind)
    rtype = (r if r is not None else out) or np.float16
    x = torch.full((rows, width), float("nan"), dtype=torch.float16, device="cuda")
    o = torch.full((rows, width), float("nan"), dtype=torch.float32 if rtype == np.float32 else torch.float16, device="cuda")
    lbm.lb_norm(x=x, out=o, kind=kind, post=post, scale=scale, eps=eps, **{n: _dev(v) for n, v in a.items()})
    torch.cuda.synchronize()
    (u, tu), (n, tn) = cacheref.norm(kind, post=post, scale=scale, eps=float(np.float32(eps)), **a)
    what = f"rows={rows} width={width} {kind} post={post} gate={gate}"
    assert_within(o.cpu().numpy(), u, cacheref.rounded(u, tu, rtype), what + " out")
    assert_within(x.cpu().numpy(), n, cacheref.rounded(n, tn, np.float16), what + " x")


WIDTHS = [1, 7, 8, 9, 64, 511, 512, 513, 1031, 2048, 2049, 4096, 4099, 8192, 8200, 16384, 16391, 32768]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(lbm, width, kind):
    say(f"[case] norm width={width} {kind}")
    rng = np.random.default_rng(width)
    if width == 1 and kind == "layer":
        return _run(lbm, rng, 5, 1, kind="layer", eps=0.5)  # the variance is 0
    for rows in (1, 6):
        _run(lbm, rng, rows, width, kind=kind, post=width > 1, gate="rows", scale=0.7)


@pytest.mark.parametrize("y,r,out", [(np.float16, np.float16, None), (np.float32, np.float16, None), (np.float32, np.float32, None),
                                     (np.float16, None, np.float32), (np.float32, None, np.float16), (None, np.float32, None),
                                     (None, np.float16, None)])
@pytest.mark.parametrize("affine", [True, False])
def test_parts(lbm, y, r, out, affine):
    say(f"[case] norm parts y={y} r={r}")
    rng = np.random.default_rng(3)
    for gate in (None, "vector", "rows") if y is not None else (None,):
        _run(lbm, rng, 9, 1000, y=y, r=r, out=out, affine=affine, gate=gate, post=y is not None and affine, scale=-1.5)


def test_outputs_may_be_missing(lbm):
    torch = lbtest.torch_dev()
    say("[case] norm one output")
    r = torch.randn((4, 96), device="cuda")
    y = torch.randn((4, 96), device="cuda").half()
    x, o = torch.empty_like(y), torch.empty_like(r)
    lbm.lb_norm(r, x=x, y=y, out=o)
    x2, o2 = torch.zeros_like(x), torch.zeros_like(o)
    lbm.lb_norm(r, x=x2, y=y)
    lbm.lb_norm(r, y=y, out=o2)
    assert torch.equal(x, x2) and torch.equal(o, o2)


def test_many_rows_and_large_values(lbm):
    say("[case] norm 3000 rows")
    rng = np.random.default_rng(5)
    _run(lbm, rng, 3000, 256, kind="layer", gate="vector")
    data = _inputs(rng, 64, 777, np.float32, np.float32, True, False, None, "layer")
    data["r"] += np.float32(300)  # far from 0: the variance is about the mean
    _run(lbm, rng, 64, 777, kind="layer", y=np.float32, data=data)


def test_zero_rows_and_nan_rows_stay_apart(lbm):
    torch = lbtest.torch_dev()
    say("[case] norm NaN rows")
    r = torch.randn((7, 300), device="cuda")
    r[2] = 0
    r[3, 5] = float("nan")
    r[5, 7] = float("inf")
    x = torch.empty((7, 300), dtype=torch.float16, device="cuda")
    lbm.lb_norm(r, x=x)
    assert (x[2] == 0).all() and x[3].isnan().all() and x[5, 7].isnan() and (x[5, :7] == 0).all()
    good = [0, 1, 4, 6]
    want = torch.empty((4, 300), dtype=torch.float16, device="cuda")
    lbm.lb_norm(r[good].contiguous(), x=want)
    assert torch.equal(x[good], want)
    for t in (x[:0], torch.empty((0, 300), dtype=torch.float16, device="cuda")):
        lbm.lb_norm(r[:0], x=t)


@pytest.mark.parametrize("width", [63, 1000, 3001])
def test_strides_alignments_and_in_place(lbm, width):
    """Column blocks of one buffer at odd offsets, and outputs in the place of inputs."""
    torch = lbtest.torch_dev()
    say(f"[case] norm strides width={width}")
    rows = 11
    buf = torch.randn((rows, 3 * width + 5), device="cuda").half()
    y, r, x = buf[:, 1: 1 + width], buf[:, 1 + width: 1 + 2 * width], buf[:, 2 + 2 * width: 2 + 3 * width]
    keep = buf.clone()
    w = torch.randn(width, device="cuda").half()
    want_x, want_o = torch.empty((rows, width), dtype=torch.float16, device="cuda"), torch.empty((rows, width), dtype=torch.float16, device="cuda")
    lbm.lb_norm(r.contiguous(), x=want_x, y=y.contiguous(), out=want_o, weight=w, kind="layer")
    lbm.lb_norm(r, x=x, y=y, out=r, weight=w, kind="layer")  # r in place
    assert torch.equal(x, want_x) and torch.equal(r, want_o) and torch.equal(y, keep[:, 1: 1 + width])
    assert torch.equal(buf[:, 0], keep[:, 0]) and torch.equal(buf[:, 1 + 2 * width], keep[:, 1 + 2 * width])
    buf.copy_(keep)
    lbm.lb_norm(r, x=y, y=y, out=r, weight=w, kind="layer")  # both in place
    assert torch.equal(y, want_x) and torch.equal(r, want_o)


def test_refusals(lbm):
    torch = lbtest.torch_dev()
    say("[case] norm refusals")
    r = torch.randn((4, 64), device="cuda")
    x = torch.empty((4, 64), dtype=torch.float16, device="cuda")
    for kw in (dict(r=None), dict(kind="batch"), dict(weight=x[0].float()), dict(weight=x[0, :63]), dict(x=x[:3]), dict(x=r),
               dict(out=x), dict(y=r.double()), dict(gate=x[:2]), dict(x=x.cpu()), dict(y=x[:, ::2])):
        with pytest.raises(ValueError):
            lbm.lb_norm(**{"r": r, "x": x, **kw})
    for kw in (dict(eps=-1.0), dict(post_weight=x[0]), dict(x=None), dict(weight=x[1])):
        with pytest.raises(lbm.LBError):
            lbm.lb_norm(**{"r": r, "x": x, **kw})


def test_graph_and_stream(lbm):
    torch = lbtest.torch_dev()
    say("[case] norm graph")
    r, y = torch.zeros((5, 2100), device="cuda"), torch.zeros((5, 2100), device="cuda").half()
    x, o = torch.empty_like(y), torch.empty_like(r)
    lbm.lb_norm(r, x=x, y=y, out=o, post=True)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lbm.lb_norm(r, x=x, y=y, out=o, post=True)
    side = torch.cuda.Stream()
    for i in range(3):
        r.normal_()
        y.normal_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        x2, o2 = torch.empty_like(y), torch.empty_like(r)
        torch.cuda.synchronize()
        lbm.lb_norm(r, x=x2, y=y, out=o2, post=True, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(x, x2) and torch.equal(o, o2)
