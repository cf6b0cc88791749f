"""lb_route and lb_route_combine against plain float64 references, and a mixture layer of all four calls."""
import math

import numpy as np
import pytest

import lb_synth
from tests import bankref, lbtest
from tests.bankref import assert_within
from tests.lbtest import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


def _check(r, logits, k, renorm, what):
    ids, w, off, token, row = bankref.route(logits, k, renorm)
    assert np.array_equal(r.experts.cpu().numpy(), ids), f"{what}: experts"
    assert np.array_equal(r.offsets.cpu().numpy(), off), f"{what}: offsets"
    assert np.array_equal(r.token.cpu().numpy(), token), f"{what}: token"
    assert np.array_equal(r.row.cpu().numpy(), row), f"{what}: row"
    # the argument of exp is off by half a step of its size (at most max|z - top|), exp by two steps, the sum of up to
    # `experts` terms by as many and the quotient by one
    z = np.where(np.isfinite(logits.astype(np.float64)), logits.astype(np.float64), 0.0)
    steps = 2 * np.abs(z).max(initial=0.0) + 2 + logits.shape[1] + 2
    got = r.weights.cpu().numpy().astype(np.float64)
    assert (np.abs(got - w) <= 2.0 ** -24 * 2 * steps * w + 2.0 ** -149).all(), f"{what}: weights"


@pytest.mark.parametrize("tokens", [1, 2, 15, 64, 65, 129, 1000])
@pytest.mark.parametrize("experts,k", [(1, 1), (2, 2), (8, 2), (64, 6), (65, 64), (130, 1), (300, 7), (1024, 5)])
def test_route(lbm, tokens, experts, k):
    say(f"[case] route tokens={tokens} experts={experts} k={k}")
    rng = np.random.default_rng(tokens * 1000 + experts)
    for dt in (np.float32, np.float16):
        z = (rng.standard_normal((tokens, experts)) * 2).astype(dt)
        for renorm in (True, False):
            r = lbm.Route(tokens, experts, k, renormalise=renorm).run(lbtest.to_dev(z))
            _check(r, z, k, renorm, f"{dt.__name__} renorm={renorm}")


@pytest.mark.parametrize("tokens", [7, 200])
def test_route_special_values(lbm, tokens):
    """Ties, signed zeros, masked experts, NaN, infinities, rows with nothing to choose."""
    say(f"[case] route special tokens={tokens}")
    rng = np.random.default_rng(tokens)
    z = rng.integers(-2, 3, (tokens, 12)).astype(np.float32)  # many ties
    z[0] = -np.inf
    z[1] = np.nan
    z[2] = [0.0, -0.0] * 6
    z[3, 2:] = -np.inf
    z[4, 5] = np.inf
    z[5, [1, 7]] = np.inf
    z[6] = np.finfo(np.float32).min
    z[6, 3] = -np.inf
    r = lbm.Route(tokens, 12, 4)
    r.run(lbtest.to_dev(z))
    _check(r, z, 4, True, "special")
    with np.errstate(over="ignore"):
        z16 = z.astype(np.float16)  # the lowest number becomes -inf
    r.run(lbtest.to_dev(z16))
    _check(r, z16, 4, True, "special fp16")


def test_route_many_tokens(lbm):
    say("[case] route 20000 tokens")
    z = np.random.default_rng(1).standard_normal((20000, 16)).astype(np.float16)
    z[:, 5] = 9  # one expert takes a row of every token
    r = lbm.Route(20000, 16, 2).run(lbtest.to_dev(z))
    _check(r, z, 2, True, "20000 tokens")


def test_route_no_tokens(lbm):
    torch = lbtest.torch_dev()
    say("[case] route no tokens")
    r = lbm.Route(0, 8, 2)
    r.offsets.fill_(7)
    r.run(torch.empty((0, 8), dtype=torch.float32, device="cuda"))
    torch.cuda.synchronize()
    assert (r.offsets == 0).all()


def test_route_strided_logits(lbm):
    torch = lbtest.torch_dev()
    say("[case] route strided")
    base = torch.randn((90, 37), device="cuda")
    z = base[:, 3:19]
    _check(lbm.Route(90, 16, 3).run(z), z.cpu().numpy(), 3, True, "strided")


@pytest.mark.parametrize("tokens", [5, 300])
def test_route_in_a_graph(lbm, tokens):
    torch = lbtest.torch_dev()
    say(f"[case] route graph tokens={tokens}")
    z = torch.empty((tokens, 16), device="cuda")
    r = lbm.Route(tokens, 16, 3)
    inputs = [torch.randn((tokens, 16), device="cuda") for _ in range(3)]
    z.copy_(inputs[0])
    r.run(z)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.run(z)
    for v in inputs:
        z.copy_(v)
        r.token.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _check(r, v.cpu().numpy(), 3, True, "replay")


# ---------------------------------------------------------------- combine
def _combine(lbm, tokens, k, width, residual, out, y_rows=None, pad=(0, 0, 0), off=0, drop=True):
    torch = lbtest.torch_dev()
    rng = np.random.default_rng(width + tokens)
    y_rows = tokens * k if y_rows is None else y_rows
    y = rng.standard_normal((y_rows, width)).astype(np.float16)
    row = rng.integers(0, max(y_rows, 1), (tokens, k)).astype(np.int32)
    if drop:
        row[rng.random((tokens, k)) < 0.2] = -1
        row[0, 0] = y_rows
        row[-1, -1] = 2 ** 31 - 1
    w = rng.standard_normal((tokens, k)).astype(np.float32)
    r = rng.standard_normal((tokens, width)).astype(out) if residual else None
    dt = torch.float16 if out == np.float16 else torch.float32

    def strided(v, ld, t):
        b = torch.full((v.shape[0] * ld + 16,), 5.0, dtype=t, device="cuda")
        view = b[off:off + v.shape[0] * ld].view(v.shape[0], ld)[:, :width]
        view.copy_(lbtest.to_dev(v))
        return b, view

    _, yd = strided(y, width + pad[0], torch.float16)
    rd = strided(r, width + pad[1], dt)[1] if residual else None
    ob, od = strided(np.full((tokens, width), 5.0, out), width + pad[2], dt)
    lbm.lb_route_combine(yd, lbtest.to_dev(row), lbtest.to_dev(w), od, residual=rd)
    torch.cuda.synchronize()
    ref, size = np.zeros((tokens, width)), np.zeros((tokens, width))
    for j in range(k):
        ok = (row[:, j] >= 0) & (row[:, j] < y_rows)
        part = w[ok, j, None].astype(np.float64) * y[row[ok, j]].astype(np.float64)
        ref[ok] += part
        size[ok] += np.abs(part)
    if residual:
        ref += r.astype(np.float64)
        size += np.abs(r.astype(np.float64))
    tol = 2.0 ** -24 * (k + 1) * size  # a rounding of each partial sum
    assert_within(od.cpu().numpy(), ref, tol + bankref.HALF[out] * (np.abs(ref) + tol) + bankref.TINY[out], "combine")
    mask = torch.ones_like(ob, dtype=torch.bool)
    mask[off:off + od.shape[0] * od.stride(0)].view(od.shape[0], -1)[:, :width] = False
    assert (ob[mask] == 5.0).all(), "wrote outside out's rows"


@pytest.mark.parametrize("tokens,k,width", [(1, 1, 1), (1, 2, 4096), (5, 3, 257), (300, 8, 600), (33, 64, 8), (70, 2, 2056)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("out", [np.float16, np.float32])
def test_combine(lbm, tokens, k, width, residual, out):
    say(f"[case] combine tokens={tokens} k={k} width={width}")
    _combine(lbm, tokens, k, width, residual, out)
    _combine(lbm, tokens, k, width, residual, out, pad=(8, 16, 24))
    _combine(lbm, tokens, k, width, residual, out, pad=(3, 1, 5), off=1)


def test_combine_in_place_and_empty(lbm):
    torch = lbtest.torch_dev()
    say("[case] combine in place, no rows")
    y = torch.randn((6, 64), device="cuda").half()
    row = torch.tensor([[0, 5], [-1, 2]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 2.0], [1.0, -1.0]], device="cuda")
    out = torch.randn((2, 64), device="cuda")
    want = out.double() + torch.stack([0.5 * y[0].double() + 2 * y[5].double(), -y[2].double()])
    lbm.lb_route_combine(y, row, w, out, residual=out)
    torch.cuda.synchronize()
    assert (out.double() - want).abs().max() <= 2.0 ** -24 * 4 * 16
    _combine(lbm, 4, 2, 64, True, np.float32, y_rows=0, drop=False)


def test_combine_refusals(lbm):
    torch = lbtest.torch_dev()
    say("[case] combine and route refusals")
    y, out = torch.zeros((4, 64), dtype=torch.float16, device="cuda"), torch.zeros((2, 64), device="cuda")
    row, w = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.zeros((2, 2), device="cuda")
    for bad in (lambda: lbm.lb_route_combine(y.float(), row, w, out), lambda: lbm.lb_route_combine(y[:, :63], row, w, out),
                lambda: lbm.lb_route_combine(y, row.long(), w, out), lambda: lbm.lb_route_combine(y, row, w.half(), out),
                lambda: lbm.lb_route_combine(y, row, w[:1], out), lambda: lbm.lb_route_combine(y, row, w, out.cpu()),
                lambda: lbm.lb_route_combine(y, row, w, out, residual=out.half()),
                lambda: lbm.Route(4, 8, 2).run(torch.zeros((4, 9), device="cuda")),
                lambda: lbm.Route(4, 8, 2).run(torch.zeros((5, 8), device="cuda")),
                lambda: lbm.Route(4, 8, 2).run(torch.zeros((4, 8), device="cuda").double()),
                lambda: lbm.Route(4, 8, 2).run(torch.zeros((4, 8)))):
        with pytest.raises(ValueError):
            bad()


# ------------------------------------------------------------- all together
@pytest.mark.parametrize("tokens", [1, 9, 400])
def test_mixture_layer(lbm, tokens):
    """route -> gate and up projections by expert -> down projections by expert -> combine, with the residual stream.

    Each stage is checked on its own inputs; the whole against float64 with every stage's relative error (fp16
    intermediates: half a step each) carried along in the 2-norm.
    """
    torch = lbtest.torch_dev()
    say(f"[case] mixture layer tokens={tokens}")
    d, f, s, n, k = 256, 352, 24, 8, 2
    up = [lb_synth.layer_inputs(d, f, s, True, seed=81, layer=e) for e in range(n)]
    gate = [lb_synth.layer_inputs(d, f, s, True, seed=82, layer=e) for e in range(n)]
    down = [lb_synth.layer_inputs(f, d, s, True, seed=83, layer=e) for e in range(n)]
    mk = lambda ps: [lbm.Layer.from_paths(p) for p in ps]  # noqa: E731
    first, second = lbm.Bank(mk(up), mk(gate)), lbm.Bank(mk(down))
    x = lb_synth.activations(tokens, d, seed=5)
    z = np.random.default_rng(6).standard_normal((tokens, n)).astype(np.float32)
    z[:, 3] = -np.inf
    xd, zd = lbtest.to_dev(x), lbtest.to_dev(z)
    r = lbm.Route(tokens, n, k)
    h = torch.empty((tokens * k, f), dtype=torch.float16, device="cuda")
    o = torch.empty((tokens * k, d), dtype=torch.float16, device="cuda")
    stream = lbtest.to_dev(x.astype(np.float32))
    out = torch.empty_like(stream)

    def run():
        r.run(zd)
        first.grouped(xd, r.offsets, h, index=r.token, act="silu")
        second.grouped(h, r.offsets, o)
        r.combine(o, out, residual=stream)

    run()
    torch.cuda.synchronize()
    _check(r, z, k, True, "routing")
    ids, w, off, token, row = bankref.route(z, k, True)
    hh, oo = h.cpu().numpy(), o.cpu().numpy()
    for e in range(n):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        ref, tol = bankref.fused(x[token[lo:hi]], up[e], gate[e], "silu")
        assert_within(hh[lo:hi], ref, tol, f"gate and up of expert {e}")
        ref, tol = bankref.fused(hh[lo:hi], down[e])
        assert_within(oo[lo:hi], ref, tol, f"down of expert {e}")
    ref = x.astype(np.float64).copy()
    for t in range(tokens):
        for j in range(k):
            e = ids[t, j]
            v, _ = bankref.fused(x[t:t + 1], up[e], gate[e], "silu")
            ref[t] += w[t, j] * bankref.fused(v.astype(np.float16), down[e])[0][0]
    rel = np.linalg.norm(out.cpu().numpy() - ref) / np.linalg.norm(ref)
    assert rel <= 2 * 2.0 ** -11 + math.sqrt(d) * 2.0 ** -24, rel
    # the same in a graph, replayed
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        out.zero_()
        h.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    first.close()
    second.close()
