"""A decoder layer of all calls together: norms, LittleBit projections (banks), the 8-bit cache and attention over it, for
prompts and then token by token, eager and captured.

Every stage is held against float64 on the numbers that the GPU had before it, so each has its own tolerance."""
import numpy as np
import pytest

import lb_synth
from tests import bankref, cacheref, lbtest
from tests.lbtest import say

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, INNER, RANK, PAGE = 256, 8, 2, 40, 384, 48, 16
EPS = 1e-5


@pytest.fixture(scope="module")
def lbm():
    lbtest.torch_dev()
    return lbtest.ensure_built()


class Layer:
    """One decoder layer: x += attention(norm(x)); x += down(silu(gate(n)) * up(n)), n = norm(x), with a norm of the
    attention's output as well."""

    def __init__(self, lbm, rows, rope):
        torch = lbtest.torch_dev()
        self.lbm, self.rope = lbm, rope
        f = lambda a, b, k: lb_synth.layer_inputs(a, b, RANK, True, seed=77, layer=k)  # noqa: E731
        self.paths = {"qkv": f(HIDDEN, (HEADS + 2 * KV) * DIM, 0), "out": f(HEADS * DIM, HIDDEN, 1), "up": f(HIDDEN, INNER, 2),
                      "gate": f(HIDDEN, INNER, 3), "down": f(INNER, HIDDEN, 4)}
        made = {n: lbm.Layer.from_paths(p) for n, p in self.paths.items()}
        self.bank = {n: lbm.Bank([made[n]]) for n in ("qkv", "out", "down")}
        self.bank["mlp"] = lbm.Bank([made["up"]], [made["gate"]])
        for bank in self.bank.values():
            bank.reserve(rows)
        rng = np.random.default_rng(5)
        self.weights = {n: (1 + 0.2 * rng.standard_normal(HIDDEN)).astype(np.float16) for n in ("before", "post", "mlp")}
        self.w = {n: lbtest.to_dev(v) for n, v in self.weights.items()}
        half = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
        self.x = torch.zeros((rows, HIDDEN), device="cuda")  # the residual stream, fp32
        self.n1, self.n2, self.o = half(rows, HIDDEN), half(rows, HIDDEN), half(rows, HIDDEN)
        self.qkv, self.att, self.inner = half(rows, (HEADS + 2 * KV) * DIM), half(rows, HEADS * DIM), half(rows, INNER)
        self.mid, self.y = torch.zeros_like(self.x), torch.zeros_like(self.x)

    def parts(self):
        q, k = HEADS * DIM, KV * DIM
        return self.qkv[:, :q], self.qkv[:, q: q + k], self.qkv[:, q + k:]

    def run(self, cache, lengths, table, start=None):
        self.lbm.lb_norm(self.x, x=self.n1, weight=self.w["before"], eps=EPS)
        self.bank["qkv"].forward(self.n1, self.qkv)
        q, k, v = self.parts()
        cache.append(k, v, lengths, table, start=start, q=q, q_out=q, rope=self.rope)  # q turned in place
        cache.attend(q, self.att, lengths, table, start=start)
        self.bank["out"].forward(self.att, self.o)
        self.lbm.lb_norm(self.x, x=self.n2, y=self.o, out=self.mid, post=True, post_weight=self.w["post"], weight=self.w["mlp"], eps=EPS)
        self.bank["mlp"].forward(self.n2, self.inner, act="silu")
        self.bank["down"].forward(self.inner, self.y, residual=self.mid)

    def outputs(self):
        return [t.clone() for t in (self.n1, self.qkv, self.att, self.o, self.mid, self.n2, self.inner, self.y)]


def _host(t):
    return t.cpu().numpy()


def _cache_numbers(cache, ref, lengths, table):
    """Puts into the reference what the library's cache holds (a rotated number next to a border may be a step off):
    reading is exact to a sixteenth of a step, so the numbers can be told from it."""
    torch = lbtest.torch_dev()
    n = int(lengths.sum())
    k, v = (torch.empty((n, KV * DIM), dtype=torch.float16, device="cuda") for _ in range(2))
    start = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    cache.read(k, v, lbtest.to_dev(lengths), lbtest.to_dev(table), start=lbtest.to_dev(start))
    for name, got in (("k", _host(k)), ("v", _host(v))):
        for b in range(len(lengths)):
            for p in range(lengths[b]):
                page, off = table[b, p // PAGE], p % PAGE
                s = ref.scale[name][page].astype(np.float64)[:, None]
                number = got[start[b] + p].astype(np.float64).reshape(KV, DIM) / np.where(s > 0, s, 1.0)
                assert np.abs(number - np.rint(number)).max() < 0.07 and np.abs(np.rint(number) - ref.num[name][page, off]).max() <= 1
                ref.num[name][page, off] = np.rint(number)


def _check(layer, cache, ref, x, lengths, table, start, new, what):
    n1, qkv, att, o, mid, n2, inner, y = map(_host, layer.outputs())
    w = layer.weights
    _, (want, tol) = cacheref.norm("rms", r=x, weight=w["before"], eps=EPS)
    cacheref.assert_within(n1, want, cacheref.rounded(want, tol, np.float16), what + " first norm")
    want, tol = bankref.fused(n1, layer.paths["qkv"])
    q, k = HEADS * DIM, KV * DIM
    bankref.assert_within(qkv[:, q:], want[:, q:], tol[:, q:], what + " k and v")
    rope, at = _host(layer.rope), 0
    for b in range(len(new)):
        for i in range(new[b]):
            p = lengths[b] - new[b] + i
            turned = cacheref.turn(want[at, :q].reshape(HEADS, DIM), p, rope, False).ravel()
            # projection and rotation round to fp16 each: the pair's tolerances, then half a step
            t = np.abs(tol[at, :q]).reshape(HEADS, DIM).max(1).repeat(DIM) * 1.5
            assert (np.abs(qkv[at, :q] - turned) <= t + 2.0 ** -11 * np.abs(turned) + 2.0 ** -24).all(), what + " q"
            at += 1
    ref.append(qkv[:, q: q + k], qkv[:, q + k:], lengths, table, start, rope)
    _cache_numbers(cache, ref, lengths, table)
    want, tol = cacheref.attend(ref, qkv[:, :q], lengths, table, start)
    cacheref.assert_within(att, want, tol + 2.0 ** -20 * np.abs(want), what + " attention")
    want, tol = bankref.fused(att, layer.paths["out"])
    bankref.assert_within(o, want, tol, what + " output projection")
    (want, tol), (want2, tol2) = cacheref.norm("rms", r=x, y=o, post=True, post_weight=w["post"], weight=w["mlp"], eps=EPS)
    cacheref.assert_within(mid, want, cacheref.rounded(want, tol, np.float32), what + " residual")
    cacheref.assert_within(n2, want2, cacheref.rounded(want2, tol2, np.float16), what + " second norm")
    want, tol = bankref.fused(n2, layer.paths["up"], layer.paths["gate"], "silu")
    bankref.assert_within(inner, want, tol, what + " feed-forward")
    want, tol = bankref.fused(inner, layer.paths["down"], residual=mid, out=np.float32)
    bankref.assert_within(y, want, tol, what + " layer")


def test_prompt_then_tokens(lbm):
    torch = lbtest.torch_dev()
    rng = np.random.default_rng(1)
    prompts, steps, columns = [21, 40, 7], 20, 5
    rope = lbtest.to_dev(cacheref.rope_table(columns * PAGE, DIM))
    table = rng.permutation(3 * columns).reshape(3, columns).astype(np.int32)
    tdev = lbtest.to_dev(table)
    ref = cacheref.Cache(3 * columns, PAGE, KV, DIM)
    cache, twin = (lbm.Cache(3 * columns, PAGE, KV, DIM) for _ in range(2))
    cache.reserve(3, HEADS, 3, columns * PAGE)
    say("[case] decoder layer, prompts")
    layer = Layer(lbm, sum(prompts), rope)
    x = rng.standard_normal((sum(prompts), HIDDEN)).astype(np.float32)
    layer.x.copy_(lbtest.to_dev(x))
    lengths, start = np.array(prompts, np.int32), np.array([0, 21, 61, 68], np.int32)
    for c in (twin, cache):
        layer.run(c, lbtest.to_dev(lengths), tdev, lbtest.to_dev(start))
    torch.cuda.synchronize()
    _check(layer, cache, ref, x, lengths, table, start, prompts, "prompt")

    say("[case] decoder layer, tokens")
    eager, graph = Layer(lbm, 3, rope), Layer(lbm, 3, rope)
    ldev = torch.zeros(3, dtype=torch.int32, device="cuda")
    ldev.copy_(lbtest.to_dev(lengths + 1))
    for g in (eager, graph):
        g.x.copy_(lbtest.to_dev(rng.standard_normal((3, HIDDEN)).astype(np.float32)))
    torch.cuda.synchronize()
    captured = torch.cuda.CUDAGraph()
    with torch.cuda.graph(captured):
        graph.run(cache, ldev, tdev)
    for i in range(steps):
        say(f"[case] decoder layer, token {i}")
        x = rng.standard_normal((3, HIDDEN)).astype(np.float32)
        for g in (eager, graph):
            g.x.copy_(lbtest.to_dev(x))
        now = (lengths + 1 + i).astype(np.int32)
        ldev.copy_(lbtest.to_dev(now))
        captured.replay()
        eager.run(twin, ldev, tdev)
        torch.cuda.synchronize()
        for a, b in zip(eager.outputs(), graph.outputs()):
            assert torch.equal(a, b), f"token {i}: captured and eager differ"
        _check(graph, cache, ref, x, now, table, None, [1, 1, 1], f"token {i}")
