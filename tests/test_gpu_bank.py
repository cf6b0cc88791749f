"""lb_bank_forward and lb_bank_grouped against the float64 oracle, element by element (tolerances: tests/bankref.py)."""
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


_cache = {}


def _layers(lbm, a, b, s, residual, n, seed):
    """n layers and their paths (kept: several tests share a shape)."""
    key = (a, b, s, residual, n, seed)
    if key not in _cache:
        paths = [lb_synth.layer_inputs(a, b, s, residual, seed=seed, layer=e) for e in range(n)]
        _cache[key] = paths, [lbm.Layer.from_paths(p) for p in paths]
    return _cache[key]


def _extras(rng, n, b, rows, bias, gate_bias, residual, out):
    f = lambda *shape: rng.standard_normal(shape)  # noqa: E731
    return ((0.5 * f(n, b)).astype(np.float16) if bias else None,
            (0.5 * f(n, b)).astype(np.float16) if gate_bias else None, f(rows, b).astype(out) if residual else None)


def _dev(v):
    return None if v is None else lbtest.to_dev(v)


def _forward(lbm, a, b, s, res, M, gated=False, act="none", bias=False, residual=False, out=np.float16, seed=1):
    torch = lbtest.torch_dev()
    rng = np.random.default_rng(seed)
    up, ul = _layers(lbm, a, b, s, res, 1, 11)
    gate, gl = _layers(lbm, a, b, s, res, 1, 12) if gated else (None, None)
    bv, gv, rv = _extras(rng, 1, b, M, bias, bias and gated, residual, out)
    x = lb_synth.activations(M, a, seed=seed)
    B = lbm.Bank(ul, gl)
    y = torch.full((M, b), float("nan"), dtype=torch.float16 if out == np.float16 else torch.float32, device="cuda")
    B.forward(_dev(x), y, act=act, bias=_dev(bv), gate_bias=_dev(gv), residual=_dev(rv))
    torch.cuda.synchronize()
    ref, tol = bankref.fused(x, up[0], gate[0] if gated else None, act, bv[0] if bias else None,
                             gv[0] if gv is not None else None, rv, out)
    assert_within(y.cpu().numpy(), ref, tol, f"a={a} b={b} s={s} M={M} gated={gated} {act}")
    B.close()


SHAPES = [(1, 1, 1, False), (33, 17, 5, True), (256, 256, 32, False), (257, 129, 63, False), (1000, 600, 40, True),
          (64, 40, 300, True), (2048, 1376, 133, True)]


@pytest.mark.parametrize("a,b,s,res", SHAPES)
@pytest.mark.parametrize("M", [1, 2, 31, 32, 33, 64, 65, 200])
def test_rows(lbm, a, b, s, res, M):
    say(f"[case] bank forward a={a} b={b} s={s} M={M}")
    _forward(lbm, a, b, s, res, M)
    _forward(lbm, a, b, s, res, M, gated=True, act="silu", bias=True, residual=True, out=np.float32, seed=2)


@pytest.mark.parametrize("act", bankref.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out", [np.float16, np.float32])
def test_epilogues(lbm, act, gated, out):
    say(f"[case] bank epilogue {act} gated={gated} {out.__name__}")
    for k, (bias, residual) in enumerate(((False, False), (True, False), (False, True), (True, True))):
        _forward(lbm, 1000, 600, 40, True, 37, gated, act, bias, residual, out, seed=20 + k)


@pytest.mark.parametrize("M,b,gated", [(1024, 4000, False), (1500, 8200, False), (1100, 4100, True), (16400, 40, False),
                                       (16390, 72, True)])
def test_many_rows(lbm, M, b, gated):
    """Many rows, wide and narrow, each of them checked."""
    say(f"[case] bank forward M={M} b={b} gated={gated}")
    _forward(lbm, 128, b, 45, True, M, gated=gated, act="gelu" if not gated else "silu", bias=True, residual=True)


# the rank makes one to five column tiles per workgroup of the first product
FEW_ROWS = [(1000, 1000, 20, False), (448, 1500, 20, True), (1792, 72, 20, False), (224, 72, 60, True)]
MIDDLE = [(2112, 40, s, False) for s in (80, 190, 277, 384, 480)] + [(1100, 300, 20, True), (2112, 72, 45, True)]
MANY_NARROW = [(4200, 8200, s, True) for s in (20, 64, 95, 127, 160)]
MANY_WIDE = [(2112, 16400, s, False) for s in (20, 256, 640, 860, 1100)]


@pytest.mark.parametrize("a", [128, 131])
@pytest.mark.parametrize("M,b,s,gated", FEW_ROWS + MIDDLE + MANY_NARROW + MANY_WIDE)
def test_launch_shapes(lbm, a, M, b, s, gated):
    """Every kernel with every number of column tiles, aligned x rows and others; a sample of the rows is checked,
    the first and last of a slot among them."""
    torch = lbtest.torch_dev()
    say(f"[case] bank launch shapes a={a} M={M} b={b} s={s} gated={gated}")
    rng = np.random.default_rng(9)
    up, ul = _layers(lbm, a, b, s, gated, 1, 11)
    gate, gl = _layers(lbm, a, b, s, gated, 1, 12) if gated else (None, None)
    x = lb_synth.activations(M, a, seed=9)
    bv, _, rv = _extras(rng, 1, b, M, True, False, True, np.float32)
    B = lbm.Bank(ul, gl)
    y = torch.full((M, b), float("nan"), device="cuda")
    B.forward(_dev(x), y, act="silu", bias=_dev(bv), residual=_dev(rv))
    torch.cuda.synchronize()
    assert torch.isfinite(y).all()
    rows = np.unique(np.concatenate([[0, 15, 16, 31, 32, 63, 64, M // 64 * 64 - 1, M - 1], rng.integers(0, M, 60)]))
    ref, tol = bankref.fused(x[rows], up[0], gate[0] if gated else None, "silu", bv[0], None, rv[rows], np.float32)
    assert_within(y[torch.from_numpy(rows).cuda()].cpu().numpy(), ref, tol, f"a={a} M={M} b={b} s={s} gated={gated}")
    B.close()
    _cache.clear()


@pytest.mark.parametrize("a,M", [(2049, 5), (2743, 16), (4096, 1), (11008, 3), (28672, 1), (8192, 130)])
def test_wide_inputs(lbm, a, M):
    say(f"[case] bank forward a={a} M={M}")
    _forward(lbm, a, 96, 86, True, M, out=np.float32)


def test_windows_of_the_workspace(lbm):
    """Rank 4096 on two sides: 2 MB of latent rows per 32 rows, so 5000 rows run in windows."""
    say("[case] bank forward in windows")
    _forward(lbm, 64, 64, 4096, True, 5000, gated=True, act="none")


def test_small_and_large_values(lbm):
    """x scaled by 2^-10 and by 2^8: the latent vector keeps its bits (a linear layer scales exactly)."""
    torch = lbtest.torch_dev()
    say("[case] bank forward, scaled inputs")
    a, b, s, M = 1000, 600, 40, 40
    up, ul = _layers(lbm, a, b, s, True, 1, 11)
    B = lbm.Bank(ul)
    x = lb_synth.activations(M, a, seed=5)
    for scale in (2.0 ** -10, 2.0 ** 8):
        xs = (x.astype(np.float64) * scale).astype(np.float16)
        y = torch.empty((M, b), dtype=torch.float32, device="cuda")
        B.forward(_dev(xs), y)
        torch.cuda.synchronize()
        ref, tol = bankref.fused(xs, up[0], out=np.float32)
        assert_within(y.cpu().numpy(), ref, tol, f"scale {scale}")
    B.close()


@pytest.mark.parametrize("off,ldx,ldy,ldr", [(0, 1008, 608, 616), (1, 1003, 601, 603), (0, 1001, 600, 600), (8, 1016, 616, 600)])
@pytest.mark.parametrize("out", [np.float16, np.float32])
@pytest.mark.parametrize("M", [9, 45, 8200, 33000])
def test_strides_and_alignment(lbm, off, ldx, ldy, ldr, out, M):
    """Row strides, and x, y and residual that begin inside an allocation; what lies between y's rows stays."""
    torch = lbtest.torch_dev()
    say(f"[case] bank strides off={off} ldx={ldx} ldy={ldy} ldr={ldr} M={M}")
    a, b = 1000, 600
    up, ul = _layers(lbm, a, b, 40, True, 1, 11)
    B = lbm.Bank(ul)
    rng = np.random.default_rng(3)
    x = lb_synth.activations(M, a, seed=6)
    r = rng.standard_normal((M, b)).astype(out)
    dt = torch.float16 if out == np.float16 else torch.float32
    xb = torch.full((M * ldx + 16,), float("nan"), dtype=torch.float16, device="cuda")
    xv = xb[off:off + M * ldx].view(M, ldx)[:, :a]
    xv.copy_(_dev(x))
    rb = torch.zeros(M * ldr + 16, dtype=dt, device="cuda")
    rv = rb[off:off + M * ldr].view(M, ldr)[:, :b]
    rv.copy_(_dev(r))
    yb = torch.full((M * ldy + 16,), 7.0, dtype=dt, device="cuda")
    yv = yb[off:off + M * ldy].view(M, ldy)[:, :b]
    B.forward(xv, yv, residual=rv)
    torch.cuda.synchronize()
    ref, tol = bankref.fused(x, up[0], residual=r, out=out)
    assert_within(yv.cpu().numpy(), ref, tol, "strided")
    mask = torch.ones_like(yb, dtype=torch.bool)
    mask[off:off + M * ldy].view(M, ldy)[:, :b] = False
    assert (yb[mask] == 7.0).all(), "wrote outside y's rows"
    B.close()


def test_residual_in_place(lbm):
    torch = lbtest.torch_dev()
    say("[case] bank residual in place")
    a, b, M = 1000, 600, 70
    up, ul = _layers(lbm, a, b, 40, True, 1, 11)
    B = lbm.Bank(ul)
    x = lb_synth.activations(M, a, seed=7)
    r = np.random.default_rng(4).standard_normal((M, b)).astype(np.float32)
    y = _dev(r)
    B.forward(_dev(x), y, residual=y)
    torch.cuda.synchronize()
    ref, tol = bankref.fused(x, up[0], residual=r, out=np.float32)
    assert_within(y.cpu().numpy(), ref, tol, "in place")
    B.close()


@pytest.mark.parametrize("M", [12, 300, 8200, 33000])
def test_rows_are_independent(lbm, M):
    """NaN and infinity in one row of x stay in that row's output (each launch shape)."""
    torch = lbtest.torch_dev()
    say(f"[case] bank NaN rows M={M}")
    a, b = 1000, 600
    up, ul = _layers(lbm, a, b, 40, True, 1, 11)
    B = lbm.Bank(ul)
    x = lb_synth.activations(M, a, seed=8)
    clean = torch.empty((M, b), dtype=torch.float16, device="cuda")
    B.forward(_dev(x), clean)
    x[3, 5], x[M - 3, 999] = np.nan, np.inf
    y = torch.empty_like(clean)
    B.forward(_dev(x), y)
    torch.cuda.synchronize()
    keep = [i for i in range(M) if i not in (3, M - 3)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[M - 3]).any()
    B.close()


# ------------------------------------------------------------------ grouped
def _counts(kind, n, rng):
    if kind == "one has all":
        c = np.zeros(n, int)
        c[n // 2] = 133
    elif kind == "one row each":
        c = np.ones(n, int)
    elif kind == "ragged":
        c = rng.integers(0, 70, n)
        c[0] = c[-1] = 0
        c[1 % n] = 64
    elif kind == "large":
        c = rng.integers(100, 400, n)
        c[n // 3] = 0
    else:
        c = np.zeros(n, int)
    return c


def _grouped(lbm, a, b, s, res, n, counts, gated=False, act="none", bias=False, residual=False, out=np.float16,
             gather=False, before=0, behind=0, seed=1):
    torch = lbtest.torch_dev()
    rng = np.random.default_rng(seed)
    up, ul = _layers(lbm, a, b, s, res, n, 31)
    gate, gl = _layers(lbm, a, b, s, res, n, 32) if gated else (None, None)
    off = before + np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(off[-1]) + behind
    bv, gv, rv = _extras(rng, n, b, rows, bias, bias and gated, residual, out)
    xr = max(1, rows // 3) if gather else max(rows, 1)
    x = lb_synth.activations(xr, a, seed=seed)
    index = rng.integers(0, xr, rows).astype(np.int32) if gather else None
    B = lbm.Bank(ul, gl)
    y = torch.full((rows, b), 9.0, dtype=torch.float16 if out == np.float16 else torch.float32, device="cuda")
    B.grouped(_dev(x), _dev(off), y, index=_dev(index), act=act, bias=_dev(bv), gate_bias=_dev(gv), residual=_dev(rv))
    torch.cuda.synchronize()
    got = y.cpu().numpy()
    for e in range(n):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        xe = x[index[lo:hi]] if gather else x[lo:hi]
        ref, tol = bankref.fused(xe, up[e], gate[e] if gated else None, act, bv[e] if bias else None,
                                 gv[e] if gv is not None else None, rv[lo:hi] if residual else None, out)
        assert_within(got[lo:hi], ref, tol, f"expert {e} of {n}, rows {lo}..{hi}")
    assert (got[:before] == 9.0).all() and (got[off[-1]:] == 9.0).all(), "wrote rows of no expert"
    B.close()


@pytest.mark.parametrize("kind", ["none", "one has all", "one row each", "ragged"])
@pytest.mark.parametrize("n", [1, 2, 8, 65])
def test_grouped_counts(lbm, kind, n):
    say(f"[case] grouped n={n} {kind}")
    c = _counts(kind, n, np.random.default_rng(n))
    _grouped(lbm, 200, 136, 21, True, n, c, before=3, behind=5)
    _grouped(lbm, 200, 136, 21, True, n, c, gated=True, act="silu", bias=True, residual=True, out=np.float32,
             gather=True, behind=2, seed=2)


@pytest.mark.parametrize("gated", [False, True])
def test_grouped_large(lbm, gated):
    say(f"[case] grouped large gated={gated}")
    c = _counts("large", 9, np.random.default_rng(5))
    _grouped(lbm, 128, 8200, 45, True, 9, c, gated=gated, act="gelu_tanh", bias=True, gather=True)


@pytest.mark.parametrize("gated", [False, True])
def test_grouped_many_rows(lbm, gated):
    """64-row slots: runs of none, one, a slot less a row, a slot, a slot and a row, and long ones."""
    say(f"[case] grouped many rows gated={gated}")
    c = np.array([0, 1, 63, 64, 65, 700, 0, 1151, 131])
    _grouped(lbm, 128, 16400, 45, False, 9, c, gated=gated, act="silu", bias=True, gather=True, before=3, behind=7)


def test_grouped_odd(lbm):
    say("[case] grouped odd sizes")
    c = _counts("ragged", 5, np.random.default_rng(6))
    _grouped(lbm, 259, 131, 63, False, 5, c, act="gelu", bias=True, residual=True, gather=True)


@pytest.mark.parametrize("b,rows", [(136, 6), (136, 1100), (8200, 1100), (16400, 2200)])
def test_grouped_index_out_of_range_reads_zeros(lbm, b, rows):
    """In each launch shape; the rows around the bad ones keep their values."""
    torch = lbtest.torch_dev()
    say(f"[case] grouped bad index rows={rows}")
    up, ul = _layers(lbm, 200, b, 21, True, 2, 31)
    B = lbm.Bank(ul)
    x = lb_synth.activations(4, 200, seed=1)
    index = np.arange(rows, dtype=np.int32) % 4
    bad = [1, rows // 2 - 1, rows // 2, rows - 1]
    index[bad] = [-1, 4, 2 ** 31 - 1, -2 ** 31]
    half = rows // 2
    y = torch.full((rows, b), 9.0, dtype=torch.float16, device="cuda")
    B.grouped(_dev(x), _dev(np.array([0, half, rows], np.int32)), y, index=_dev(index))
    torch.cuda.synchronize()
    got = y.cpu().numpy()
    assert (got[bad] == 0).all()
    for e, lo, hi in ((0, 0, half), (1, half, rows)):
        good = np.array([i for i in range(lo, hi) if i not in bad])
        ref, tol = bankref.fused(x, up[e])
        assert_within(got[good], ref[index[good]], tol[index[good]], f"good rows of expert {e}")
    B.close()


@pytest.mark.parametrize("rows", [300, 40000])
def test_grouped_many_experts(lbm, rows):
    """1024 experts (three layers over and over), some without rows, one with a third of them."""
    torch = lbtest.torch_dev()
    say(f"[case] 1024 experts rows={rows}")
    up, ul = _layers(lbm, 40, 24, 9, False, 3, 91)
    n = 1024
    rng = np.random.default_rng(rows)
    c = rng.multinomial(rows - rows // 3, np.ones(n) / n)
    c[700] += rows // 3
    off = np.concatenate([[0], np.cumsum(c)]).astype(np.int32)
    x = lb_synth.activations(rows, 40, seed=2)
    B = lbm.Bank([ul[e % 3] for e in range(n)])
    y = torch.empty((rows, 24), dtype=torch.float32, device="cuda")
    B.grouped(_dev(x), _dev(off), y)
    torch.cuda.synchronize()
    got = y.cpu().numpy()
    expert = np.repeat(np.arange(n), c)
    for k in range(3):
        mine = expert % 3 == k
        ref, tol = bankref.fused(x[mine], up[k], out=np.float32)
        assert_within(got[mine], ref, tol, f"layer {k}")
    B.close()


def test_grouped_strided_x_with_rows_to_spare(lbm):
    """x as a column slice, with more rows than the call has; a bank of one layer."""
    torch = lbtest.torch_dev()
    say("[case] grouped strided x")
    up, ul = _layers(lbm, 200, 136, 21, True, 1, 31)
    B = lbm.Bank(ul)
    base = torch.full((50, 230), float("nan"), dtype=torch.float16, device="cuda")
    xh = lb_synth.activations(50, 200, seed=4)
    x = base[:, 17:217]
    x.copy_(_dev(xh))
    y = torch.full((33, 136), 9.0, dtype=torch.float16, device="cuda")
    B.grouped(x, _dev(np.array([2, 31], np.int32)), y)
    torch.cuda.synchronize()
    got = y.cpu().numpy()
    ref, tol = bankref.fused(xh[2:31], up[0])
    assert_within(got[2:31], ref, tol, "strided x")
    assert (got[:2] == 9).all() and (got[31:] == 9).all()
    B.close()


def test_grouped_offsets_are_clamped(lbm):
    """Offsets outside [0, rows] count as their nearest value; nothing outside y is touched."""
    torch = lbtest.torch_dev()
    say("[case] grouped clamped offsets")
    up, ul = _layers(lbm, 200, 136, 21, True, 2, 31)
    B = lbm.Bank(ul)
    x = lb_synth.activations(40, 200, seed=1)
    yb = torch.full((60, 136), 9.0, dtype=torch.float16, device="cuda")
    y = yb[10:50]
    B.grouped(_dev(x), _dev(np.array([-5, 33, 2 ** 31 - 1], np.int32)), y)
    torch.cuda.synchronize()
    got = yb.cpu().numpy()
    assert (got[:10] == 9).all() and (got[50:] == 9).all()
    for e, lo, hi in ((0, 0, 33), (1, 33, 40)):
        ref, tol = bankref.fused(x[lo:hi], up[e])
        assert_within(got[10 + lo:10 + hi], ref, tol, f"expert {e}")
    B.close()


def test_grouped_and_forward_agree(lbm):
    """The same rows through lb_bank_grouped and, expert by expert, lb_bank_forward: both within the tolerance of the
    float64 result (the calls choose their kernels by their own row counts, so sums may be ordered differently)."""
    torch = lbtest.torch_dev()
    say("[case] grouped and forward")
    up, ul = _layers(lbm, 200, 136, 21, True, 8, 31)
    B = lbm.Bank(ul)
    c = np.array([3, 0, 32, 33, 1, 0, 20, 8])
    off = np.concatenate([[0], np.cumsum(c)]).astype(np.int32)
    xh = lb_synth.activations(int(off[-1]), 200, seed=3)
    x = _dev(xh)
    y = torch.empty((int(off[-1]), 136), dtype=torch.float16, device="cuda")
    z = torch.empty_like(y)
    B.grouped(x, _dev(off), y, act="silu")
    for e in range(8):
        lo, hi = int(off[e]), int(off[e + 1])
        if hi > lo:
            B.forward(x[lo:hi], z[lo:hi], expert=e, act="silu")
    torch.cuda.synchronize()
    for e in range(8):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            ref, tol = bankref.fused(xh[lo:hi], up[e], act_name="silu")
            assert_within(y[lo:hi].cpu().numpy(), ref, tol, f"grouped, expert {e}")
            assert_within(z[lo:hi].cpu().numpy(), ref, tol, f"forward, expert {e}")
    B.close()


# ------------------------------------------------------------------ use
@pytest.mark.parametrize("M", [1, 40, 300])
def test_graph_replays(lbm, M):
    """Captured forward and grouped calls, replayed with new inputs and eager work between, equal eager results."""
    torch = lbtest.torch_dev()
    say(f"[case] bank graph M={M}")
    up, ul = _layers(lbm, 200, 136, 21, True, 4, 31)
    B = lbm.Bank(ul)
    B.reserve(M)
    off = _dev(np.array([0, M // 3, M // 3, M // 2, M], np.int32))
    x = torch.empty((M, 200), dtype=torch.float16, device="cuda")
    y, z = (torch.empty((M, 136), dtype=torch.float16, device="cuda") for _ in range(2))

    def run():
        B.forward(x, y, expert=2, act="silu")
        B.grouped(x, off, z)

    inputs = [_dev(lb_synth.activations(M, 200, seed=50 + i)) for i in range(3)]
    want = []
    for v in inputs:
        x.copy_(v)
        run()
        torch.cuda.synchronize()
        want.append((y.clone(), z.clone()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for v, (wy, wz) in zip(inputs, want):
        x.copy_(v)
        y.zero_()
        z.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, wy) and torch.equal(z, wz)
    B.close()


def test_capture_beyond_the_reservation_is_refused(lbm):
    torch = lbtest.torch_dev()
    say("[case] bank capture beyond reservation")
    _, ul = _layers(lbm, 200, 136, 21, True, 1, 31)
    B = lbm.Bank(ul)
    B.reserve(8)
    x = torch.zeros((4096, 200), dtype=torch.float16, device="cuda")
    y = torch.empty((4096, 136), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.capture_begin()
        try:
            with pytest.raises(lbm.LBError) as ei:
                B.forward(x, y)
            B.forward(x[:8], y[:8])
        finally:
            g.capture_end()
    assert ei.value.status == lbm.LB_ENOTREADY
    y.fill_(3)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert (y[:8] == 0).all() and (y[8:] == 3).all()
    B.close()


def test_growth_keeps_captured_calls_valid(lbm):
    torch = lbtest.torch_dev()
    say("[case] bank growth after capture")
    up, ul = _layers(lbm, 200, 136, 21, True, 1, 31)
    B = lbm.Bank(ul)
    xh = lb_synth.activations(40, 200, seed=9)
    x, y = _dev(xh), torch.empty((40, 136), dtype=torch.float16, device="cuda")
    B.forward(x, y)
    torch.cuda.synchronize()
    want = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.forward(x, y)
    big = torch.zeros((5000, 200), dtype=torch.float16, device="cuda")
    B.forward(big, torch.empty((5000, 136), dtype=torch.float16, device="cuda"))
    for _ in range(2):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    B.close()


def test_two_banks_on_two_streams(lbm):
    torch = lbtest.torch_dev()
    say("[case] two banks, two streams")
    _, la = _layers(lbm, 200, 136, 21, True, 1, 31)
    _, lc = _layers(lbm, 1000, 600, 40, True, 1, 11)
    banks = [lbm.Bank(la), lbm.Bank(lc)]
    xs = [_dev(lb_synth.activations(100, B.a, seed=1)) for B in banks]
    want = [torch.empty((100, B.b), dtype=torch.float16, device="cuda") for B in banks]
    for B, x, w in zip(banks, xs, want):
        B.forward(x, w, act="gelu")
    outs = [[torch.empty_like(w) for _ in range(8)] for w in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(8):
        for k in range(2):
            banks[k].forward(xs[k], outs[k][i], act="gelu", stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        for o in outs[k]:
            assert torch.equal(o, want[k])
    for B in banks:
        B.close()


def test_repacked_layers_are_seen(lbm):
    """Signs and scales set again after the bank was made are the ones it uses."""
    torch = lbtest.torch_dev()
    say("[case] bank after repacking")
    old = lb_synth.layer_inputs(200, 136, 21, True, seed=71)
    new = lb_synth.layer_inputs(200, 136, 21, True, seed=72)
    L = lbm.Layer.from_paths(old)
    B = lbm.Bank([L])
    for i, p in enumerate(new):
        lbm.lb_pack_signs(L.handle, i, p["su"], p["sv"])
        lbm.lb_set_scales(L.handle, i, p["h"], p["g"], p["l"])
    x = lb_synth.activations(5, 200, seed=1)
    y = torch.empty((5, 136), dtype=torch.float16, device="cuda")
    B.forward(_dev(x), y)
    torch.cuda.synchronize()
    ref, tol = bankref.fused(x, new[0:2])
    assert_within(y.cpu().numpy(), ref, tol, "repacked")
    B.close()
    L.close()


def test_refusals(lbm):
    torch = lbtest.torch_dev()
    say("[case] bank refusals")
    _, ul = _layers(lbm, 200, 136, 21, True, 2, 31)
    _, other = _layers(lbm, 1000, 600, 40, True, 1, 11)
    with pytest.raises(lbm.LBError):
        lbm.Bank(ul + other)
    with pytest.raises(ValueError):
        lbm.Bank(ul, ul[:1])
    unset = lbm.Layer(200, 136, 21, True)
    with pytest.raises(lbm.LBError) as ei:
        lbm.Bank([unset])
    assert ei.value.status == lbm.LB_ENOTREADY
    B = lbm.Bank(ul)
    f16, cuda = torch.float16, "cuda"
    x, y = torch.zeros((4, 200), dtype=f16, device=cuda), torch.full((4, 136), 5.0, dtype=f16, device=cuda)
    off = torch.zeros(3, dtype=torch.int32, device=cuda)
    for bad in (lambda: B.forward(x[:3], y), lambda: B.forward(x[:, :199], y), lambda: B.forward(x.float(), y),
                lambda: B.forward(x, y[:, :100]), lambda: B.forward(x, y, act="tanh"),
                lambda: B.forward(x, y, bias=y[0]), lambda: B.forward(x, y, residual=y.float()),
                lambda: B.forward(x, y, residual=y[:2]), lambda: B.forward(x.cpu(), y), lambda: B.forward(x, y.cpu()),
                lambda: B.forward(x.t().contiguous().t(), y), lambda: B.grouped(x, off[:2], y),
                lambda: B.grouped(x, off.long(), y), lambda: B.grouped(x, off, y, index=off)):
        with pytest.raises(ValueError):
            bad()
    assert lbm.lb_bank_shape(B.handle) == (2, False, 200, 136, torch.cuda.current_device())
    B.device += 1  # tensors of another GPU than the bank's
    with pytest.raises(ValueError):
        B.forward(x, y)
    B.device -= 1
    lib, p = lbm.load_library(), y.data_ptr()
    base = dict(e=0, x=x.data_ptr(), ldx=200, y=p, ldy=136, yt=0, M=4, act=0, bias=None, gb=None, res=None, ldr=0)
    for bad in (dict(e=2), dict(e=-1), dict(x=None), dict(y=None), dict(ldx=199), dict(ldy=135), dict(yt=2), dict(M=-1),
                dict(M=1 << 31), dict(act=5), dict(act=-1), dict(gb=x.data_ptr()), dict(res=x.data_ptr(), ldr=100),
                dict(x=p), dict(x=p + 64), dict(res=p + 2, ldr=136), dict(res=p, ldr=137), dict(bias=p), dict(x=p + 1),
                dict(y=p + 2, yt=1), dict(ldx=1 << 33)):
        assert lib.lb_bank_forward(B.handle, *{**base, **bad}.values(), None) == lbm.LB_EINVAL, bad
    # without an index x needs all rows
    assert lib.lb_bank_grouped(B.handle, x.data_ptr(), 3, 200, None, off.data_ptr(), 4, p, 136, 0, 0, None, None, None, 0,
                               None) == lbm.LB_EINVAL
    assert lib.lb_bank_forward(B.handle, 0, None, 200, None, 136, 0, 0, 0, None, None, None, 0, None) == lbm.LB_OK
    torch.cuda.synchronize()
    assert (y == 5.0).all()
    B.close()
