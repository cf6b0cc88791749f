"""Inputs and outputs that are column blocks of one buffer: they share no element, so they are no overlap."""
import numpy as np
import pytest

import lb_synth
from tests import bankref, lbtest
from tests.bankref import assert_within
from tests.lbtest import say

pytestmark = pytest.mark.gpu

A, Bw = 200, 136


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


@pytest.fixture(scope="module")
def layers(lbm):
    paths = [lb_synth.layer_inputs(A, Bw, 21, True, seed=31, layer=e) for e in range(2)]
    return paths, [lbm.Layer.from_paths(p) for p in paths]


@pytest.mark.parametrize("M", [1, 5, 700, 2000])
@pytest.mark.parametrize("first", ["x", "y"])
def test_x_and_y_of_one_buffer(lbm, layers, M, first):
    torch = lbtest.torch_dev()
    say(f"[case] x and y of one buffer M={M}")
    paths, ul = layers
    bank = lbm.Bank(ul)
    buf = torch.full((M, A + Bw), 7.0, dtype=torch.float16, device="cuda")
    x, y = (buf[:, :A], buf[:, A:]) if first == "x" else (buf[:, Bw:], buf[:, :Bw])
    xh = lb_synth.activations(M, A, seed=3)
    x.copy_(lbtest.to_dev(xh))
    ref, tol = bankref.fused(xh, paths[1])
    bank.forward(x, y, expert=1)
    torch.cuda.synchronize()
    assert_within(y.cpu().numpy(), ref, tol, "forward")
    y.fill_(7)
    bank.grouped(x, lbtest.to_dev(np.array([0, 0, M], np.int32)), y)
    torch.cuda.synchronize()
    assert_within(y.cpu().numpy(), ref, tol, "grouped")
    assert np.array_equal(x.cpu().numpy(), xh), "x was written"
    bank.close()


@pytest.mark.parametrize("out", [np.float16, np.float32])
def test_residual_and_y_of_one_buffer(lbm, layers, out):
    torch = lbtest.torch_dev()
    say(f"[case] residual and y of one buffer {out.__name__}")
    paths, ul = layers
    bank = lbm.Bank(ul)
    M = 90
    buf = torch.zeros((M, 2 * Bw + 3), dtype=torch.float16 if out == np.float16 else torch.float32, device="cuda")
    r, y = buf[:, Bw + 3:], buf[:, :Bw]
    rh = np.random.default_rng(1).standard_normal((M, Bw)).astype(out)
    r.copy_(lbtest.to_dev(rh))
    xh = lb_synth.activations(M, A, seed=4)
    bank.forward(lbtest.to_dev(xh), y, residual=r)
    torch.cuda.synchronize()
    ref, tol = bankref.fused(xh, paths[0], residual=rh, out=out)
    assert_within(y.cpu().numpy(), ref, tol, "forward")
    assert np.array_equal(r.cpu().numpy(), rh) and (buf[:, Bw:Bw + 3] == 0).all()
    with pytest.raises(lbm.LBError):  # one column in common
        bank.forward(lbtest.to_dev(xh), y, residual=buf[:, Bw - 1:2 * Bw - 1])
    bank.close()


def test_combine_within_one_buffer(lbm):
    torch = lbtest.torch_dev()
    say("[case] combine within one buffer")
    t, w = 40, 72
    buf = torch.randn((t, 3 * w), device="cuda").half()
    y, r, o = buf[:, :w], buf[:, w:2 * w], buf[:, 2 * w:]
    row = torch.randint(0, t, (t, 2), device="cuda", dtype=torch.int32)
    weights = torch.randn((t, 2), device="cuda")
    part = y.double()[row.long()] * weights.double().unsqueeze(2)
    want, size = r.double() + part.sum(1), r.double().abs() + part.abs().sum(1)
    lbm.lb_route_combine(y, row, weights, o, residual=r)
    torch.cuda.synchronize()
    # a rounding of each of three partial sums in fp32, and that of the result
    tol = 3 * 2.0 ** -24 * size
    assert ((o.double() - want).abs() <= tol + 2.0 ** -11 * (want.abs() + tol) + 2.0 ** -25).all()
    with pytest.raises(lbm.LBError):
        lbm.lb_route_combine(y, row, weights, buf[:, w - 1:2 * w - 1])
