"""Row scales of every size: the latent vector keeps its 22 bits whatever |h| is, in the kernels of every row count."""
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


def _run(lbm, up, gate, x, b):
    torch = lbtest.torch_dev()
    ul = [lbm.Layer.from_paths(up)]
    gl = [lbm.Layer.from_paths(gate)] if gate else None
    B = lbm.Bank(ul, gl)
    y = torch.full((x.shape[0], b), float("nan"), device="cuda")
    B.forward(lbtest.to_dev(x), y)
    torch.cuda.synchronize()
    got = y.cpu().numpy().astype(np.float64)
    B.close()
    for L in ul + (gl or []):
        L.close()
    return got


def _sparse(M, a, rng):
    """Rows with a single number of 11 bits in them."""
    x = np.zeros((M, a), np.float16)
    x[np.arange(M), rng.integers(0, a, M)] = rng.integers(1025, 2048, M) * rng.choice([-1.0, 1.0], M) / 1024
    return x


def _exact_paths(a, b, h, paths, seed):
    """Rank 1, g = 1 and l of 11 bits: with rows of _sparse w = l t is a product of two 11-bit numbers, which the two
    halves of a latent number hold exactly, so what is left are the roundings of the second product's sums."""
    rng = np.random.default_rng(seed)
    out = []
    for p in range(paths):
        d = lb_synth.path_inputs(a, b, 1, seed, path=p)
        d["g"] = np.ones(a, np.float16)
        d["l"] = np.array([rng.integers(1025, 2048) / 1024], np.float16)
        d["h"] = h[p]
        out.append(d)
    return out


def _exact(x, paths):
    """y in float64 (33-bit products) and the largest error of fp32 sums: hi and lo of every path add a rounding of a
    partial sum each and joining them another, a whole step (2^-23) for each, as the rounding of a matrix product's
    sum is not stated."""
    y = oracle.forward(x, paths)
    w = oracle.latent(x, paths)
    size = sum(np.abs(np.outer(w[:, p], d["h"].astype(np.float64))) for p, d in enumerate(paths))
    return y, (2 * len(paths) + 1) * 2.0 ** -23 * size


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("top", [0, -3, -6, -9, -12, -15])
def test_exact_latent_numbers(lbm, M, top):
    """h in [2^(top - 2), 2^(top + 1)): one path, two (the second's h of another size), and gated."""
    say(f"[case] exact latent numbers M={M} h=2^{top}")
    a, b = 8, 40
    rng = np.random.default_rng(100 - top)
    x = _sparse(M, a, rng)
    scale = lambda t: (rng.uniform(1, 2, b) * 2.0 ** rng.integers(t - 2, t + 1, b)).astype(np.float16)  # noqa: E731
    one = _exact_paths(a, b, [scale(top)], 1, 1)
    two = _exact_paths(a, b, [scale(top), scale(top // 2)], 2, 2)
    far = _exact_paths(a, b, [scale(top), scale(8)], 2, 3)
    last = _exact_paths(a, b, [scale(8), scale(top)], 2, 3)
    last[0]["l"][:] = 0
    for paths, name in ((one, "one path"), (two, "two paths"), (far, "paths of far sizes"), (last, "the second path alone")):
        ref, tol = _exact(x, paths)
        assert_within(_run(lbm, paths, None, x, b), ref, tol + 2.0 ** -149, name)
    v, tv = _exact(x, one)
    for gate in (one, _exact_paths(a, b, [scale(2)], 1, 4)):
        g, tg = _exact(x, gate)
        tol = np.abs(v) * tg + np.abs(g) * tv + tv * tg + 2.0 ** -24 * np.abs(v * g) + 2.0 ** -149
        assert_within(_run(lbm, one, gate, x, b), v * g, tol, "gated")


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("gated", [False, True])
def test_scales_of_many_sizes(lbm, M, gated):
    """h spread over 2^-15 .. 2^3 within one layer, some of them zero, l raised to match."""
    say(f"[case] scales of many sizes M={M} gated={gated}")
    a, b, s = 16, 40, 8

    def layer(seed):
        rng = np.random.default_rng(seed)
        paths = lb_synth.layer_inputs(a, b, s, True, seed=seed)
        for d in paths:
            d["h"] = (2.0 ** rng.uniform(-15, 3, b)).astype(np.float16)
            d["h"][rng.integers(0, b, 3)] = 0
            d["l"] = (d["l"].astype(np.float64) * 64).astype(np.float16)
        return paths

    up, gate = layer(5), layer(6) if gated else None
    x = lb_synth.activations(M, a, seed=3)
    ref, tol = bankref.fused(x, up, gate, out=np.float32)
    assert_within(_run(lbm, up, gate, x, b), ref, tol, f"M={M} gated={gated}")


@pytest.mark.parametrize("M", ROWS)
def test_layers_from_real_weights(lbm, M):
    """Layers as the initialisation makes them: h of a few hundredths."""
    say(f"[case] layers from real weights M={M}")
    a, b, s = 96, 80, 12
    up, gate = (oracle.dual_svid(lb_synth.weight_matrix(a, b, seed), s, True) for seed in (3, 4))
    for d in up + gate:
        d.update(a=a, b=b, s=s)
    x = lb_synth.activations(M, a, seed=4)
    for g in (None, gate):
        ref, tol = bankref.fused(x, up, g, out=np.float32)
        assert_within(_run(lbm, up, g, x, b), ref, tol, f"M={M} gated={g is not None}")
