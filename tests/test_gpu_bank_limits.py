"""The range of the latent vector: 22 bits from 2^-14 to fp16's largest number, 2^-36 below, no finite y above."""
import numpy as np
import pytest

import lb_synth
import oracle
from tests import bankref, lbtest
from tests.bankref import assert_within
from tests.lbtest import say

pytestmark = pytest.mark.gpu

#: row counts whose slots have 16, 32 and 64 rows in the narrow layers of these tests
ROWS = [300, 4100, 65600]


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


def _layer(a, b, l, seed=1):
    """Rank 1, g = 1: w = +-l x for a row x with one number in it."""
    d = lb_synth.path_inputs(a, b, 1, seed)
    d["g"], d["l"] = np.ones(a, np.float16), np.array([l], np.float16)
    return [d]


def _run(lbm, paths, x, gate=None):
    torch = lbtest.torch_dev()
    layers = [lbm.Layer.from_paths(p) for p in ([paths] if gate is None else [paths, gate])]
    B = lbm.Bank(layers[:1], layers[1:] or None)
    y = torch.zeros((x.shape[0], paths[0]["b"]), device="cuda")
    B.forward(lbtest.to_dev(x), y)
    torch.cuda.synchronize()
    got = y.cpu().numpy().astype(np.float64)
    B.close()
    for L in layers:
        L.close()
    return got


def _rows(M, a, values, rng):
    x = np.zeros((M, a), np.float16)
    x[np.arange(M), rng.integers(0, a, M)] = values
    return x


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("gated", [False, True])
def test_largest_latent_numbers(lbm, M, gated):
    """|w| up to 65504 is exact; 65536 and more give no finite y, in their own rows alone."""
    say(f"[case] largest latent numbers M={M} gated={gated}")
    a, b = 8, 40
    rng = np.random.default_rng(M)
    paths = _layer(a, b, 16)
    gate = _layer(a, b, 2.0 ** -4, seed=2) if gated else None  # w <= 2^8 on that side
    # 16 x for x of 11 bits reaches 65504 = 16 4094 and 65536 = 16 4096
    v = rng.choice([1.0, 1000.0, 4092.0, 4094.0, 4096.0, 5000.0, 60000.0], M)
    x = _rows(M, a, v, rng)
    got = _run(lbm, paths, x, gate)
    fits = v < 4096
    ref, size = oracle.forward(x[fits], paths), np.abs(np.outer(16 * v[fits], paths[0]["h"].astype(np.float64)))
    if gated:
        g = oracle.forward(x[fits], gate)
        ref, size = ref * g, size * np.abs(g)
    # a step for each of the two products, their joining, twice with gates, and the gate product
    assert_within(got[fits], ref, (7 if gated else 3) * 2.0 ** -23 * size, "within the range")
    assert not np.isfinite(got[~fits]).any()


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("by", [-8, -12, -16, -20, -24])
def test_small_latent_numbers(lbm, M, by):
    """w of about 2^by: off by 2^-23 of itself or 2^-36, whichever is more, and by the second product's roundings."""
    say(f"[case] small latent numbers M={M} 2^{by}")
    a, b = 8, 40
    rng = np.random.default_rng(M - by)
    paths = _layer(a, b, 2.0 ** (by // 2) * 1.37)
    v = rng.uniform(1, 2, M) * 2.0 ** (by - by // 2) * rng.choice([-1, 1], M)
    x = _rows(M, a, v.astype(np.float16), rng)
    w = oracle.latent(x, paths)
    size = np.abs(w) * np.abs(paths[0]["h"].astype(np.float64))
    # w in fp32: half a step; hi exact, lo half a step of fp16 (2^-11 of at most 2^-11 |w|) or half of its smallest
    # (2^-25 2^-11); the second product as above
    off = np.maximum(2.0 ** -22 * np.abs(w), 2.0 ** -36) * np.abs(paths[0]["h"].astype(np.float64))
    assert_within(_run(lbm, paths, x), oracle.forward(x, paths), off + 2.0 ** -24 * size + 3 * 2.0 ** -23 * size, f"2^{by}")


@pytest.mark.parametrize("rows", [300, 40000])
def test_1024_layers_and_experts_in_a_graph(lbm, rows):
    """The largest number of layers, routed and grouped, captured once and replayed on other inputs."""
    torch = lbtest.torch_dev()
    say(f"[case] 1024 layers in a graph rows={rows}")
    a, b, n, k = 40, 24, 1024, 2
    paths = [lb_synth.layer_inputs(a, b, 9, False, seed=91, layer=e) for e in range(3)]
    layers = [lbm.Layer.from_paths(p) for p in paths]
    bank = lbm.Bank([layers[e % 3] for e in range(n)])
    bank.reserve(rows * k)
    route = lbm.Route(rows, n, k)
    x, z = torch.empty((rows, a), dtype=torch.float16, device="cuda"), torch.empty((rows, n), device="cuda")
    y = torch.zeros((rows * k, b), dtype=torch.float16, device="cuda")
    out = torch.empty((rows, b), device="cuda")

    def run():
        route.run(z)
        bank.grouped(x, route.offsets, y, index=route.token)
        route.combine(y, out)

    gen = torch.Generator(device="cuda").manual_seed(rows)
    inputs, want = [], []
    for _ in range(3):
        inputs.append((torch.randn(x.shape, generator=gen, device="cuda").half(), torch.randn(z.shape, generator=gen, device="cuda")))
        x.copy_(inputs[-1][0])
        z.copy_(inputs[-1][1])
        run()
        torch.cuda.synchronize()
        want.append(out.clone())
    # the eager result itself, from the routing that lb_route returned
    ids, w = route.experts.cpu().numpy(), route.weights.double().cpu().numpy()
    dense, tols = (np.stack(v) for v in zip(*(bankref.fused(x.cpu().numpy(), p) for p in paths)))
    ref, tol = np.zeros((rows, b)), np.zeros((rows, b))
    for j in range(k):
        at = ids[:, j] % 3, np.arange(rows)
        ref += w[:, j, None] * dense[at]
        tol += w[:, j, None] * (tols[at] + 2 * 2.0 ** -24 * np.abs(dense[at]))  # and two roundings of the sum
    assert_within(want[-1].cpu().numpy(), ref, tol, "eager")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for (xi, zi), wi in zip(inputs, want):
        x.copy_(xi)
        z.copy_(zi)
        y.zero_()
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, wi)
    bank.close()
