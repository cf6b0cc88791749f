"""The activations by themselves: a layer that is the identity hands them every fp16 number exactly."""
import math

import numpy as np
import pytest

from tests import bankref, lbtest
from tests.lbtest import say

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24  # half a step of fp32


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


def _exact(v, name):
    if name == "gelu_tanh":  # (1 + tanh u) / 2 without cancellation
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    with np.errstate(over="ignore"):
        return bankref.act(v, name)


def _half_steps(v, name):
    """Roundings of half a step each, relative to the result.  exp is as far off as its argument is in absolute
    numbers: three roundings of v^2 / 2 (square, constant, product), two of v, six of 2 u; what follows, with the
    hardware's exp2 and reciprocal (a whole step each) and nine terms of a fit, makes at most sixteen."""
    if name == "gelu":
        return 16 + 3 * v * v / 2
    if name == "gelu_tanh":
        return 16 + 6 * 2 * math.sqrt(2.0 / math.pi) * np.abs(v + 0.044715 * v ** 3)
    return 16 + 2 * np.abs(v) if name == "silu" else np.zeros_like(v)


@pytest.mark.parametrize("name", bankref.ACTS)
@pytest.mark.parametrize("out", [np.float16, np.float32])
@pytest.mark.parametrize("rows", [1000, 4096, 65536])
def test_every_number(lbm, name, out, rows):
    """Every finite fp16 number through the kernels of each slot size; fp32 y within the roundings of the formula at
    hand, in the tails too, fp16 y within its own on top."""
    torch = lbtest.torch_dev()
    say(f"[case] activation {name} {out.__name__} rows={rows}")
    one = dict(a=1, b=1, s=1, su=np.ones((1, 1), np.uint32), sv=np.ones((1, 1), np.uint32), h=np.ones(1, np.float16),
               g=np.ones(1, np.float16), l=np.ones(1, np.float16))
    L = lbm.Layer.from_paths([one])
    B = lbm.Bank([L])
    x = np.arange(65536, dtype=np.uint16).view(np.float16)
    x = np.where(np.isfinite(x), x, np.float16(0)).reshape(-1, 1)
    y = torch.full((65536, 1), float("nan"), dtype=torch.float16 if out == np.float16 else torch.float32, device="cuda")
    xd = lbtest.to_dev(x)
    for lo in range(0, 65536, rows):
        B.forward(xd[lo:lo + rows], y[lo:lo + rows], act=name)
    torch.cuda.synchronize()
    got = y.cpu().numpy().astype(np.float64)[:, 0]
    v = x.astype(np.float64)[:, 0]
    ref = _exact(v, name)
    # exp2 gives 0 for what is below the smallest normal number, infinity above the largest
    tol = STEP * _half_steps(v, name) * np.abs(ref) + (np.abs(v) * 2.0 ** -125 if name not in ("none", "relu") else 0)
    if out == np.float16:
        tol = tol + bankref.HALF[out] * (np.abs(ref) + tol) + bankref.TINY[out]
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), [(v[i], got[i], ref[i], (got[i] - ref[i]) / ref[i]) for i in np.nonzero(bad)[0][:4]]
    B.close()
    L.close()
