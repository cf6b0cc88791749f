"""Measured cases of the expert-layer operators.

Four operators of a feed-forward or projection layer whose weights are LittleBit factors:

forward   y = act(layer(x) + bias) + residual, or act(gate(x) + gate_bias) * (layer(x) + bias) + residual
grouped   the same for rows sorted by expert, each expert a layer of its own, the row counts on the device
route     the top-k experts of every token, their weights, and the order of the rows by expert
combine   out[t] = residual[t] + sum_j weight[t, j] * y[row[t, j]]

where layer(x) = sum_p h_p * (S_U,p (l_p * (S_V,p^T (g_p * x)))), S_U,p and S_V,p of +-1.

With ``own`` false everything here is elementary torch arithmetic in 32 bits; with ``own`` true the calls
are those of this repository's package.
"""
import math

import torch

own = False
DEV = "cuda"

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    """Shapes: the 4096-wide projections and the 4096 -> 11008 feed-forward of the measured workloads, with
    their ranks; expert counts and token counts are generic."""
    forward = dict(op="forward", paths=2, gated=False, act="none", bias=False, residual=False, out="f16")
    grouped = dict(op="grouped", paths=2, gated=False, act="none", bias=False, residual=False, out="f16")
    return [
        # an attention output projection, one token, added to a 32-bit residual stream
        dict(forward, name="projection, 1 row", a=4096, b=4096, s=86, rows=1, residual=True, out="f32"),
        # gate and up projection of one token: latency
        dict(forward, name="gated, 1 row", a=4096, b=11008, s=133, rows=1, gated=True, act="silu"),
        # the same for a batch of sequences, at 0.3 bits a weight
        dict(forward, name="gated, 128 rows", a=4096, b=11008, s=431, rows=128, gated=True, act="silu"),
        # odd sizes throughout, one path, a biased layer with an exact GELU
        dict(forward, name="odd sizes, 1023 rows", a=1031, b=2743, s=63, rows=1023, paths=1, act="gelu", bias=True,
             residual=True),
        # a prompt through gate and up projection
        dict(forward, name="gated, 4096 rows", a=4096, b=11008, s=133, rows=4096, gated=True, act="silu"),
        # four tokens, two of eight experts each: one or two rows an expert
        dict(grouped, name="8 experts, 8 rows", a=4096, b=11008, s=133, experts=8, k=2, rows=8, gated=True, act="silu",
             gather=True),
        # many small experts with a ragged batch
        dict(grouped, name="64 experts, 1542 rows", a=1024, b=1407, s=61, experts=64, k=6, rows=1542, gated=True,
             act="gelu_tanh", bias=True, gather=True),
        # a prompt's down projection
        dict(grouped, name="8 experts, 8192 rows", a=11008, b=4096, s=133, experts=8, k=2, rows=8192, gather=False),
        # the routing of one token
        dict(op="route", name="route, 1 token", tokens=1, experts=8, k=2, renormalise=True, logits="f32"),
        # the routing of a long batch; 16-bit logits, so there are ties, some experts masked out
        dict(op="route", name="route, 16384 tokens", tokens=16384, experts=64, k=6, renormalise=True, logits="f16"),
        # a token's expert outputs joined
        dict(op="combine", name="combine, 4 tokens", tokens=4, k=2, width=4096, residual=True, out="f32"),
        # a prompt's
        dict(op="combine", name="combine, 8192 tokens", tokens=8192, k=2, width=4096, residual=True, out="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges, no dearer than the dearest of them."""
    most = max(work(c)["flops"] for c in listed())
    op = rng.choice(("forward", "forward", "grouped", "grouped", "route", "combine"))
    if op == "route":
        experts = rng.randint(2, 128)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, k=rng.randint(1, min(8, experts)),
                    renormalise=rng.random() < 0.7, logits=rng.choice(("f16", "f32")))
    if op == "combine":
        return dict(op=op, tokens=_log(rng, 1, 8192), k=rng.randint(1, 8), width=_log(rng, 256, 4096),
                    residual=rng.random() < 0.5, out=rng.choice(("f16", "f32")))
    while True:
        case = dict(op=op, paths=rng.choice((1, 2, 2)), gated=rng.random() < 0.5, act=rng.choice(ACTS),
                    bias=rng.random() < 0.4, residual=rng.random() < 0.4, out=rng.choice(("f16", "f16", "f32")))
        wide = op == "grouped"
        case |= dict(a=_log(rng, 256, 4096 if wide else 11008), b=_log(rng, 256, 4096 if wide else 11008),
                     s=_log(rng, 8, 302 if wide else 431))
        if rng.random() < 0.7:  # most widths are multiples of eight
            case |= dict(a=case["a"] // 8 * 8, b=case["b"] // 8 * 8)
        if wide:
            experts = _log(rng, 2, 64)
            k = rng.randint(1, min(6, experts))
            case |= dict(experts=experts, k=k, rows=k * _log(rng, 1, 2048), gather=rng.random() < 0.6)
        else:
            case |= dict(rows=_log(rng, 1, 4096))
        if work(case)["flops"] <= most and case.get("experts", 1) * case["s"] * (case["a"] + case["b"]) <= 5e7:
            return case


def work(case):
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        size = 2 if case["logits"] == "f16" else 4
        return {"bytes": t * e * size + t * k * 16 + 4 * (e + 1), "flops": t * e * 4}
    if case["op"] == "combine":
        t, k, w = case["tokens"], case["k"], case["width"]
        size = 2 if case["out"] == "f16" else 4
        return {"bytes": t * w * (2 * k + size * (2 if case["residual"] else 1)) + t * k * 8, "flops": 2 * t * k * w}
    a, b, s, rows = case["a"], case["b"], case["s"], case["rows"]
    used = min(case.get("experts", 1), rows)
    size = 2 if case["out"] == "f16" else 4
    layers = (2 if case["gated"] else 1) * case["paths"]
    x_rows = rows // case["k"] if case.get("gather") else rows
    read = used * (layers * (s * (a + b) / 8 + 2 * (a + b + s)) + (2 * b * (2 if case["gated"] else 1) if case["bias"] else 0))
    read += 2 * x_rows * a + (size * rows * b if case["residual"] else 0) + (4 * rows if case.get("gather") else 0)
    return {"bytes": read + size * rows * b, "flops": 2.0 * rows * layers * s * (a + b)}


# ------------------------------------------------------------------ inputs
def _type(name):
    return torch.float16 if name == "f16" else torch.float32


def _words(gen, n, rows, s):
    """Canonical sign words of n factors: rows x ceil(s / 32) words each, bit k % 32 of word k // 32 for column k."""
    w = torch.randint(-(1 << 31), 1 << 31, (n, rows, (s + 31) // 32), generator=gen, device=DEV, dtype=torch.int64)
    return w.to(torch.int32)


def _signs(words, s):
    """The words as a dense +-1 matrix in 32 bits."""
    bits = (words.unsqueeze(-1) >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
    return (bits.flatten(-2)[..., :s] * 2 - 1).float()


def _uniform(gen, *shape):
    return torch.rand(shape, generator=gen, device=DEV) + 0.5


def _weights(gen, n, case):
    """n layers: sign words [n, paths, rows, words] and 16-bit scales, as a checkpoint holds them."""
    a, b, s, p = case["a"], case["b"], case["s"], case["paths"]
    return {"su": _words(gen, n * p, b, s).view(n, p, b, -1), "sv": _words(gen, n * p, a, s).view(n, p, a, -1),
            "h": _uniform(gen, n, p, b).half(), "g": _uniform(gen, n, p, a).half(),
            "l": (_uniform(gen, n, p, s) / math.sqrt(a * s * p)).half()}


def _counts(gen, case):
    """Rows of each expert: tokens choose k different experts each, some experts far more often than others."""
    tokens, e, k = case["rows"] // case["k"], case["experts"], case["k"]
    liking = torch.randn(e, generator=gen, device=DEV) * 0.7
    noise = -torch.log(-torch.log(torch.rand((tokens, e), generator=gen, device=DEV).clamp(1e-6, 1 - 1e-6)))
    chosen = (liking + noise).topk(k, dim=1).indices.flatten()
    order = torch.sort(chosen, stable=True).indices
    counts = torch.bincount(chosen, minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    return offsets, (order // k).to(torch.int32)


def _inputs(case, seed):
    """The tensors alone, from the seed."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 13)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    if case["op"] == "route":
        logits = (normal(case["tokens"], case["experts"]) * 2).to(_type(case["logits"]))
        if case["experts"] > case["k"] and case["tokens"] > 1:  # an expert that is out of service
            logits[:, seed % case["experts"]] = -math.inf
        return {"logits": logits}
    if case["op"] == "combine":
        t, k, w = case["tokens"], case["k"], case["width"]
        st = {"y": normal(t * k, w).half(), "weights": torch.softmax(normal(t, k), 1),
              "row": torch.randperm(t * k, generator=gen, device=DEV).to(torch.int32).view(t, k)}
        if t > 1:  # a token's last choice was dropped
            st["row"][seed % t, -1] = -1
        st["residual"] = normal(t, w).to(_type(case["out"])) if case["residual"] else None
        return st
    e, rows = case.get("experts", 1), case["rows"]
    st = {"up": _weights(gen, e, case), "gate": _weights(gen, e, case) if case["gated"] else None}
    st["bias"] = (normal(e, case["b"]) * 0.5).half() if case["bias"] else None
    st["gate_bias"] = (normal(e, case["b"]) * 0.5).half() if case["bias"] and case["gated"] else None
    st["offsets"] = st["index"] = None
    if case["op"] == "grouped":
        st["offsets"], index = _counts(gen, case)
        st["index"] = index if case["gather"] else None
    st["x"] = normal(rows // case["k"] if case.get("gather") else rows, case["a"]).half()
    st["residual"] = normal(rows, case["b"]).to(_type(case["out"])) if case["residual"] else None
    return st


def _layers(lbm, w, case):
    made = []
    host = {name: v.cpu().numpy() for name, v in w.items()}
    for e in range(host["h"].shape[0]):
        layer = lbm.Layer(case["a"], case["b"], case["s"], case["paths"] == 2)
        for p in range(case["paths"]):
            lbm.lb_pack_signs(layer.handle, p, host["su"][e, p], host["sv"][e, p])
            lbm.lb_set_scales(layer.handle, p, host["h"][e, p], host["g"][e, p], host["l"][e, p])
        made.append(layer)
    return made


def _dense(w, case):
    s = case["s"]
    return {"U": _signs(w["su"], s).transpose(2, 3).contiguous(), "V": _signs(w["sv"], s),
            "h": w["h"].float(), "g": w["g"].float(), "l": w["l"].float()}


def prepare(case, seed):
    """A program keeps its weights in the form that its forward reads, so that is what differs: the packed layers of
    the package, or the signs as 32-bit matrices."""
    st = _inputs(case, seed)
    st["case"] = case
    if case["op"] == "route":
        if own:
            import binary_rank_gemv_littlebitlinear_amd as lbm
            st["route"] = lbm.Route(case["tokens"], case["experts"], case["k"], renormalise=case["renormalise"])
        return st
    if case["op"] == "combine":
        st["out"] = torch.empty((case["tokens"], case["width"]), dtype=_type(case["out"]), device=DEV)
        return st
    st["y"] = torch.empty((case["rows"], case["b"]), dtype=_type(case["out"]), device=DEV)
    up, gate = st.pop("up"), st.pop("gate")
    if own:
        import binary_rank_gemv_littlebitlinear_amd as lbm
        st["bank"] = lbm.Bank(_layers(lbm, up, case), _layers(lbm, gate, case) if gate else None)
        st["bank"].reserve(case["rows"])
    else:
        st["up"], st["gate"] = _dense(up, case), _dense(gate, case) if gate else None
        if case["op"] == "grouped":  # rows of the fullest expert: the size of the padded batch
            st["cap"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
    return st


# ------------------------------------------------------------- plain forms
def _act(v, name):
    if name == "relu":
        return torch.clamp_min(v, 0)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _layer(x, w):
    """x [experts, rows, a] -> [experts, rows, b]: both products as batches over experts and paths."""
    e, p, s, b = w["U"].shape
    z = x.unsqueeze(1) * w["g"].unsqueeze(2)
    t = torch.bmm(z.flatten(0, 1), w["V"].flatten(0, 1)) * w["l"].reshape(e * p, 1, s)
    u = torch.bmm(t, w["U"].flatten(0, 1)).view(e, p, -1, b)
    return (u * w["h"].unsqueeze(2)).sum(1)


def _products(x, st):
    case = st["case"]
    v = _layer(x, st["up"])
    if st["bias"] is not None:
        v = v + st["bias"].float().unsqueeze(1)
    if st["gate"] is None:
        return _act(v, case["act"])
    g = _layer(x, st["gate"])
    if st["gate_bias"] is not None:
        g = g + st["gate_bias"].float().unsqueeze(1)
    return _act(g, case["act"]) * v


def _plain_forward(st):
    v = _products(st["x"].float().unsqueeze(0), st)[0]
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(st["y"].dtype)


def _plain_grouped(st):
    offsets, rows, cap = st["offsets"].long(), st["case"]["rows"], st["cap"]
    x = st["x"].float()
    if st["index"] is not None:
        x = x[st["index"].long()]
    at = torch.arange(rows, device=x.device)
    expert = (at.unsqueeze(1) >= offsets[1:].unsqueeze(0)).sum(1)
    slot = expert * cap + at - offsets[expert]
    padded = torch.zeros((offsets.numel() - 1) * cap, x.shape[1], device=x.device)
    padded[slot] = x
    v = _products(padded.view(-1, cap, x.shape[1]), st).flatten(0, 1)[slot]
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(st["y"].dtype)


def _plain_route(st):
    case = st["case"]
    k, e = case["k"], case["experts"]
    logits = st["logits"].float()
    logits = torch.where(torch.isnan(logits), torch.full_like(logits, -math.inf), logits)
    ranked, order = torch.sort(logits, dim=1, descending=True, stable=True)
    kept = ranked[:, :k] > -math.inf
    ids = torch.where(kept, order[:, :k], torch.full_like(order[:, :k], -1))
    part = torch.where(ranked > -math.inf, torch.exp(ranked - ranked[:, :1]), torch.zeros_like(ranked))
    total = part[:, :k].sum(1, keepdim=True) if case["renormalise"] else part.sum(1, keepdim=True)
    weights = torch.where(kept, part[:, :k] / total, torch.zeros_like(part[:, :k]))
    flat = torch.where(ids < 0, torch.full_like(ids, e), ids).flatten()
    by_expert, place = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(e + 1, device=flat.device))
    row = torch.empty_like(place)
    row[place] = torch.arange(place.numel(), device=place.device)
    row = torch.where(flat == e, torch.full_like(row, -1), row)
    token = torch.where(by_expert == e, torch.full_like(place, -1), place // k)
    i32 = torch.int32
    return {"experts": ids.to(i32), "weights": weights, "offsets": offsets.to(i32), "token": token.to(i32),
            "row": row.view(-1, k).to(i32)}


def _plain_combine(st):
    row = st["row"].long()
    part = st["y"][row.clamp_min(0)].float() * st["weights"].unsqueeze(2)
    v = torch.where((row >= 0).unsqueeze(2), part, torch.zeros_like(part)).sum(1)
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(st["out"].dtype)


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"forward": _plain_forward, "grouped": _plain_grouped, "route": _plain_route,
                "combine": _plain_combine}[op](st)
    if op == "forward":
        st["bank"].forward(st["x"], st["y"], act=case["act"], bias=st["bias"], gate_bias=st["gate_bias"],
                           residual=st["residual"])
        return st["y"]
    if op == "grouped":
        st["bank"].grouped(st["x"], st["offsets"], st["y"], index=st["index"], act=case["act"], bias=st["bias"],
                           gate_bias=st["gate_bias"], residual=st["residual"])
        return st["y"]
    if op == "route":
        r = st["route"].run(st["logits"])
        return {"experts": r.experts, "weights": r.weights, "offsets": r.offsets, "token": r.token, "row": r.row}
    import binary_rank_gemv_littlebitlinear_amd as lbm
    lbm.lb_route_combine(st["y"], st["row"], st["weights"], st["out"], residual=st["residual"])
    return st["out"]


# ------------------------------------------------------------------- exact
def _exact_layer(x, w, e, case):
    """One layer on x [rows, a], in 64 bits, path by path from the words."""
    y = 0.0
    for p in range(case["paths"]):
        k = torch.arange(case["s"], device=x.device)
        u = (w["su"][e, p].long()[:, k // 32] >> (k % 32)) & 1
        v = (w["sv"][e, p].long()[:, k // 32] >> (k % 32)) & 1
        inner = (x * w["g"][e, p].double()) @ torch.where(v == 1, 1.0, -1.0).double()
        inner = inner * w["l"][e, p].double()
        y = y + (inner @ torch.where(u == 1, 1.0, -1.0).double().t().contiguous()) * w["h"][e, p].double()
    return y


def _exact_act(v, name):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    if name == "silu":
        return v * torch.sigmoid(v)
    return v


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(case, st["logits"])
    if case["op"] == "combine":
        out = st["residual"].double() if case["residual"] else torch.zeros(case["tokens"], case["width"], device=DEV).double()
        for j in range(case["k"]):
            here = st["row"][:, j] >= 0
            at = st["row"][here, j].long()
            out[here] += st["weights"][here, j].double().unsqueeze(1) * st["y"][at].double()
        return out
    offsets = [0, case["rows"]] if case["op"] == "forward" else st["offsets"].tolist()
    out = torch.zeros((case["rows"], case["b"]), dtype=torch.float64, device=DEV)
    for e in range(len(offsets) - 1):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        x = st["x"][lo:hi] if st["index"] is None else st["x"][st["index"][lo:hi].long()]
        v = _exact_layer(x.double(), st["up"], e, case)
        if st["bias"] is not None:
            v = v + st["bias"][e].double()
        if case["gated"]:
            g = _exact_layer(x.double(), st["gate"], e, case)
            if st["gate_bias"] is not None:
                g = g + st["gate_bias"][e].double()
            v = _exact_act(g, case["act"]) * v
        else:
            v = _exact_act(v, case["act"])
        out[lo:hi] = v if st["residual"] is None else v + st["residual"][lo:hi].double()
    return out


def _exact_route(case, logits):
    """k times the lowest index of the largest logit that is left; counts and places by comparison."""
    left = logits.double()
    top = left.max(1, keepdim=True).values
    part = torch.where(left > -math.inf, torch.exp(left - top), torch.zeros_like(left))
    t, e = left.shape
    left = left.clone()
    number = torch.arange(e, device=DEV)
    ids, weights = [], []
    for _ in range(case["k"]):
        best = left.max(1, keepdim=True).values
        at = torch.where(left == best, number, e).min(1).values
        live = best[:, 0] > -math.inf
        ids.append(torch.where(live, at, torch.full_like(at, -1)))
        weights.append(torch.where(live, part.gather(1, at[:, None])[:, 0], torch.zeros_like(part[:, 0])))
        left.scatter_(1, at[:, None], -math.inf)
    ids, weights = torch.stack(ids, 1), torch.stack(weights, 1)
    weights = weights / (weights.sum(1, keepdim=True) if case["renormalise"] else part.sum(1, keepdim=True))
    token = torch.full((t * case["k"],), -1, dtype=torch.int32, device=DEV)
    row = torch.full_like(ids, -1)
    offsets = [0]
    for x in range(e):
        where = (ids == x).nonzero()  # in the order of the tokens
        place = torch.arange(len(where), device=DEV) + offsets[-1]
        token[place] = where[:, 0].to(torch.int32)
        row[where[:, 0], where[:, 1]] = place
        offsets.append(offsets[-1] + len(where))
    return {"experts": ids.to(torch.int32), "weights": weights, "offsets": torch.tensor(offsets, dtype=torch.int32),
            "token": token, "row": row.to(torch.int32)}
