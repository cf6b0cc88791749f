"""lb_norm in every shape that it is launched in, and in windows of rows, against the float64 reference."""
import numpy as np
import pytest

from tests import cacheref, lbtest, normcases
from tests.cacheref import assert_within
from tests.lbtest import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


def _check(lbm, rng, rows, width, kind, what, post=True, gate="rows", r_type=np.float16):
    torch = lbtest.torch_dev()
    f = lambda *s: rng.standard_normal(s, dtype=np.float32)  # noqa: E731
    a = {"r": (f(rows, width) * 3).astype(r_type), "y": (f(rows, width) + np.float32(0.5)).astype(np.float16),
         "gate": None if gate is None else f(rows if gate == "rows" else 1, width).astype(np.float16)}
    for name in ("weight", "bias") + (("post_weight", "post_bias") if post else ()):
        a[name] = (f(width) * np.float32(0.3) + np.float32(name.endswith("weight"))).astype(np.float16)
    x = torch.full((rows, width), float("nan"), dtype=torch.float16, device="cuda")
    o = torch.full((rows, width), float("nan"), dtype=torch.float16 if r_type is np.float16 else torch.float32, device="cuda")
    lbm.lb_norm(x=x, out=o, kind=kind, post=post, scale=0.7, **{n: None if v is None else lbtest.to_dev(v) for n, v in a.items()})
    torch.cuda.synchronize()
    (u, tu), (n, tn) = cacheref.norm(kind, post=post, scale=0.7, eps=float(np.float32(1e-5)), **a)
    assert_within(o.cpu().numpy(), u, cacheref.rounded(u, tu, r_type), what + " out")
    assert_within(x.cpu().numpy(), n, cacheref.rounded(n, tn, np.float16), what + " x")


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("shape,rows,width", normcases.CALLS)
def test_shapes(lbm, shape, rows, width, kind):
    say(f"[case] norm {shape}: {rows} x {width} {kind}")
    rng = np.random.default_rng(rows + width)
    _check(lbm, rng, rows, width, kind, f"{shape}: {rows} x {width} {kind}")
    _check(lbm, rng, rows, width, kind, f"{shape}: {rows} x {width} {kind}, no post", post=False, gate="vector", r_type=np.float32)


@pytest.mark.parametrize("width", [16, 9])
def test_windows_of_rows(lbm, width):
    """More rows than a launch takes."""
    say(f"[case] norm 2^20 + 3 rows of {width}")
    _check(lbm, np.random.default_rng(width), (1 << 20) + 3, width, "layer", f"2^20 + 3 rows of {width}")
