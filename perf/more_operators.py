"""Measured cases of what a decoder layer does between its projections.

norm     the end of a block and the beginning of the next: r' = scale * r + gate * norm(y), x = norm(r')
append   new keys and values into a paged cache of 8-bit numbers with a scale for each page and head, rotated by
         their positions on the way (queries too), and the values that the cache then holds
attend   attention over that cache, for single tokens, prompts and mixtures of both

With ``own`` false everything here is elementary torch arithmetic in 32 bits (64 for the 8-bit rounding); with ``own``
true the calls are those of this repository's package.
"""
import math
import random

import torch

own = False
DEV = "cuda"


def listed():
    """Widths and heads: the 4096- and 8192-wide models of the measured workloads (32 heads of 128, 64 of 128 that share
    8 key heads); pages, batches and lengths are generic."""
    norm = dict(op="norm", kind="rms", post=False, gate="none", scale=1.0, y="f16", r="f32", affine=True, first=False)
    append = dict(op="append", heads=64, kv_heads=8, dim=128, rot=128, interleaved=False, chunk=1)
    attend = dict(op="attend", heads=64, kv_heads=8, dim=128, chunk=1, causal=True, window=0)
    return [
        # a token between attention and feed-forward: latency
        dict(norm, name="norm, 1 row", rows=1, width=4096),
        # a prompt through a block with a norm on each side
        dict(norm, name="norm, 4096 rows, both sides", rows=4096, width=8192, post=True),
        # odd width, layer norm, a gate for every row, a scaled 16-bit residual
        dict(norm, name="norm, odd, 1023 rows", rows=1023, width=1031, kind="layer", gate="rows", scale=0.7, r="f16"),
        # one sequence's next token: latency
        dict(append, name="append, 1 token", heads=32, kv_heads=32, batch=1, longest=512, page=64),
        # the next token of a batch of sequences
        dict(append, name="append, 64 sequences", batch=64, longest=4096, page=16),
        # a prompt
        dict(append, name="append, prompt of 4096", batch=1, longest=4096, page=64, chunk=4096),
        # chunks of prompts among single tokens, partly rotated neighbouring pairs, an odd head width
        dict(append, name="append, mixed, 80 wide", heads=24, kv_heads=8, dim=80, rot=40, interleaved=True, batch=13,
             longest=1531, page=32, chunk=251),
        # one sequence's next token, a head of its own for every query: latency
        dict(attend, name="attend, 1 token", heads=32, kv_heads=32, batch=1, longest=512, page=64),
        # the next token of a batch of sequences of all lengths
        dict(attend, name="attend, 64 sequences", batch=64, longest=4096, page=16),
        # a long document's next token
        dict(attend, name="attend, 131072 keys", batch=1, longest=131072, page=128),
        # a prompt
        dict(attend, name="attend, prompt of 4096", heads=32, kv_heads=32, batch=1, longest=4096, page=64, chunk=4096),
        # chunks of prompts among single tokens, in a window, an odd head width
        dict(attend, name="attend, mixed, 80 wide", heads=24, kv_heads=8, dim=80, batch=23, longest=3001, page=32,
             chunk=251, window=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ones' ranges, no dearer than the dearest of its operator."""
    op = rng.choice(("norm", "append", "append", "attend", "attend", "attend"))
    known = [work(c) for c in listed() if c["op"] == op]
    most = {m: max(w[m] for w in known) for m in ("bytes", "flops")}
    while True:
        if op == "norm":
            case = dict(op=op, rows=_log(rng, 1, 4096), width=_log(rng, 64, 8192), kind=rng.choice(("rms", "layer")),
                        post=rng.random() < 0.4, gate=rng.choice(("none", "none", "vector", "rows")),
                        scale=rng.choice((1.0, 1.0, 0.5, 1.25)), y=rng.choice(("f16", "f32")),
                        r=rng.choice(("f16", "f32")), affine=rng.random() < 0.8, first=rng.random() < 0.15)
            if rng.random() < 0.6:
                case["width"] = (case["width"] + 7) // 8 * 8
        else:
            kv = rng.choice((1, 2, 4, 8, 8, 16, 32))
            case = dict(op=op, kv_heads=kv, heads=kv * rng.choice((1, 1, 2, 3, 4, 8)), batch=_log(rng, 1, 64),
                        dim=rng.choice((64, 72, 80, 96, 128, 128, 128, 192, 256)), page=rng.choice((16, 32, 64, 128)))
            single = rng.random() < 0.5
            case |= dict(longest=_log(rng, 1, 4096 if op == "append" or not single else 65536))
            case |= dict(chunk=1 if single else min(case["longest"], _log(rng, 2, 4096)))
            if op == "append":
                case |= dict(rot=rng.choice((case["dim"], case["dim"], case["dim"] // 4 * 2, 0)),
                             interleaved=rng.random() < 0.3)
            else:
                causal = rng.random() < 0.85
                case |= dict(causal=causal, window=_log(rng, 1, 2048) if causal and rng.random() < 0.25 else 0)
            if case["heads"] > 64 or 4 * case["batch"] * case["chunk"] * case["heads"] * case["longest"] > 4e9:
                continue
            if 4 * case["batch"] * case["longest"] * kv * case["dim"] > 2e9:
                continue
        w = work(case)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return case


def _sequences(case):
    """Tokens of each sequence and how many of them are new: the first is the longest, the others of all lengths down
    to a sixteenth; with chunks, every third sequence brings one and the others a token."""
    rng = random.Random(case["batch"] * 7919 + case["longest"] * 31 + case["chunk"])
    lengths = [case["longest"]] + [_log(rng, max(1, case["longest"] // 16), case["longest"]) for _ in range(case["batch"] - 1)]
    new = [min(n, case["chunk"]) if i % 3 == 0 else 1 for i, n in enumerate(lengths)]
    return lengths, new


def _first_read(case):
    """The tokens that the case reads back of each sequence: from the first page that has a new one."""
    lengths, new = _sequences(case)
    return [n - (n - m) // case["page"] * case["page"] for n, m in zip(lengths, new)]


def work(case):
    if case["op"] == "norm":
        t, w = case["rows"], case["width"]
        ys, rs = (2 if case["y"] == "f16" else 4), (2 if case["r"] == "f16" else 4)
        row = ys + (0 if case["first"] else rs) + rs + 2 + (2 if case["gate"] == "rows" else 0)
        return {"bytes": t * w * row + 2 * w * ((2 if case["affine"] else 0) + (1 if case["gate"] == "vector" else 0)),
                "flops": t * w * (12 if case["post"] else 8)}
    lengths, new = _sequences(case)
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        rows, back = sum(new), sum(_first_read(case))
        old = back - rows  # the tokens that share a page with new ones
        table = 4 * case["rot"] * sum(new)
        return {"bytes": rows * d * (4 * kv + 4 * h) + 2 * back * kv * d + 2 * old * kv * d + table + 4 * back * kv * d,
                "flops": rows * d * (12 * kv + 4 * h)}
    pairs = keys = 0
    for n, m in zip(lengths, new):
        lo = n - m  # the first new token
        for i in range(m):
            last = lo + i + 1 if case["causal"] else n
            pairs += min(last, case["window"]) if case["window"] else last
        keys += min(n, case["window"] + m - 1) if case["window"] else n
    return {"bytes": keys * kv * (2 * d + 8 / case["page"]) + 4 * sum(new) * h * d, "flops": 4.0 * pairs * h * d}


# ------------------------------------------------------------------ inputs
def _type(name):
    return torch.float16 if name == "f16" else torch.float32


def _starts(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _rope(case, positions):
    """Cosines, then sines, of position * 10000^(-2i / rot), from angles in 64 bits."""
    at = torch.arange(positions, device=DEV, dtype=torch.float64)
    freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=DEV, dtype=torch.float64) / case["rot"])
    angle = at.unsqueeze(1) * freq.unsqueeze(0)
    return torch.cat([torch.cos(angle), torch.sin(angle)], 1).float()


def _inputs(case, seed):
    """The tensors alone, from the seed."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    if case["op"] == "norm":
        t, w = case["rows"], case["width"]
        channel = torch.exp(normal(w) * 0.5)  # a residual stream has channels of very different sizes
        st = {"r": None if case["first"] else (normal(t, w) * channel * 3).to(_type(case["r"]))}
        st["y"] = (normal(t, w) * channel + 0.3).to(_type(case["y"]))
        for name in ("weight", "bias", "post_weight", "post_bias"):
            st[name] = None
        if case["affine"]:
            st["weight"] = (1 + 0.2 * normal(w)).half()
            st["post_weight"] = (1 + 0.2 * normal(w)).half() if case["post"] else None
            if case["kind"] == "layer":
                st["bias"] = (0.2 * normal(w)).half()
                st["post_bias"] = (0.2 * normal(w)).half() if case["post"] else None
        st["gate"] = None
        if case["gate"] != "none":
            st["gate"] = (0.5 * normal(t if case["gate"] == "rows" else 1, w)).half()
        return st
    lengths, new = _sequences(case)
    kv, d, page = case["kv_heads"], case["dim"], case["page"]
    used = [(n + page - 1) // page for n in lengths]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    at = _starts(used)
    column = torch.arange(max(used), device=DEV)
    inside = column.unsqueeze(0) < _i32(used).unsqueeze(1)
    place = (at[:-1].unsqueeze(1) + column.unsqueeze(0)).clamp_max(pages - 1).long()
    st = {"table": torch.where(inside, order[place], torch.full_like(order[place], -1)), "pages": pages}
    gain = torch.exp(normal(2, kv * d) * 0.3)  # channels of keys and values differ in size
    old = [n - m for n, m in zip(lengths, new)]
    for name, counts in (("old", old), ("new", new)):
        rows = sum(counts)
        st["k_" + name] = normal(rows, kv * d).mul_(gain[0]).half()
        st["v_" + name] = normal(rows, kv * d).mul_(gain[1]).half()
        st["start_" + name] = _starts(counts)
    st["q"] = normal(sum(new), case["heads"] * d).half()
    st["old"], st["lengths"] = _i32(old), _i32(lengths)
    return st


def _plain_cache(st, case):
    shape = (st["pages"], case["page"], case["kv_heads"], case["dim"])
    return {"k": torch.zeros(shape, dtype=torch.int8, device=DEV), "v": torch.zeros(shape, dtype=torch.int8, device=DEV),
            "ks": torch.zeros(shape[::2], dtype=torch.float32, device=DEV),
            "vs": torch.zeros(shape[::2], dtype=torch.float32, device=DEV)}


def prepare(case, seed):
    """A serving program has the cache filled by earlier calls, so here that is done by the append of each side."""
    st = _inputs(case, seed)
    st["case"] = case
    if case["op"] == "norm":
        st["x"] = torch.empty((case["rows"], case["width"]), dtype=torch.float16, device=DEV)
        st["out"] = torch.empty((case["rows"], case["width"]), dtype=_type(case["r"]), device=DEV)
        return st
    kv, d, page = case["kv_heads"], case["dim"], case["page"]
    lengths, new = _sequences(case)
    st["start"] = st["start_new"] if case["chunk"] > 1 else None  # one row a sequence needs no starts
    st["rope"] = None
    if case["op"] == "append" and case["rot"]:
        st["rope"] = _rope(case, st["table"].shape[1] * page)
    st["interleaved"] = case.get("interleaved", False)
    if own:
        import binary_rank_gemv_littlebitlinear_amd as lbm
        st["cache"] = lbm.Cache(st["pages"], page, kv, d)
        if case["op"] == "attend":
            st["cache"].reserve(sum(new), case["heads"], len(lengths), max(lengths))
    else:
        st["cache"] = _plain_cache(st, case)
    _write(st, st["k_old"], st["v_old"], st["old"], st["start_old"])
    if case["op"] == "append":
        st["q_out"] = torch.empty_like(st["q"])
        if not own:  # a program knows the pages that it hands out
            st["touched"] = _touched(st, sum(new), st["lengths"], st["start_new"])
        back = _first_read(case)
        st["start_back"] = _starts(back)
        st["k_back"] = torch.empty((sum(back), kv * d), dtype=torch.float16, device=DEV)
        st["v_back"] = torch.empty_like(st["k_back"])
        return st
    _write(st, st["k_new"], st["v_new"], st["lengths"], st["start_new"])
    for name in ("k_old", "v_old", "k_new", "v_new"):
        del st[name]
    st["out"] = torch.empty_like(st["q"])
    st["longest"], st["most"] = max(lengths), max(new)
    return st


def _touched(st, rows, lengths, start):
    seq, pos = _rows_of(rows, lengths, start)
    return torch.unique(st["table"][seq, pos // st["case"]["page"]]).long()


def _write(st, k, v, lengths, start):
    """Appends to the cache of either side."""
    if k.shape[0] == 0:
        return
    if own:
        st["cache"].append(k, v, lengths, st["table"], start=start, rope=st["rope"], interleaved=st["interleaved"])
    else:
        _plain_append(st, k, v, None, lengths, start, _touched(st, k.shape[0], lengths, start))


# ------------------------------------------------------------- plain forms
def _plain_norm_of(v, kind, weight, bias):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5)
    if weight is not None:
        v = v * weight.float()
    return v if bias is None else v + bias.float()


def _plain_norm(st):
    case = st["case"]
    u = st["y"].float()
    if case["post"]:
        u = _plain_norm_of(u, case["kind"], st["post_weight"], st["post_bias"])
    if st["gate"] is not None:
        u = u * st["gate"].float()
    if st["r"] is not None:
        u = u + case["scale"] * st["r"].float()
    x = _plain_norm_of(u, case["kind"], st["weight"], st["bias"])
    return {"x": x.half(), "r": u.to(_type(case["r"]))}


def _rows_of(rows, lengths, start):
    """Sequence and position of every row; without starts sequence i has row i, its last token."""
    row = torch.arange(rows, device=DEV)
    if start is None:
        return row, lengths.long() - 1
    seq = torch.searchsorted(start.long(), row, right=True) - 1
    return seq, lengths.long()[seq] - (start[1:] - start[:-1]).long()[seq] + row - start.long()[seq]


def _rotate(x, pos, rope, interleaved):
    """x [rows, heads, dim] in 32 or 64 bits."""
    half = rope.shape[1] // 2
    cos, sin = (t[pos].to(x.dtype).unsqueeze(1) for t in (rope[:, :half], rope[:, half:]))
    turned, rest = x[..., : 2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, rest], -1)


def _plain_store(values, scales, x, page, off, touched):
    """x [rows, heads, dim] in 64 bits into the pages; a page that begins here forgets its scale, one whose scale grows
    has its numbers rounded again. touched: the pages of the rows, each once."""
    size = values.shape[1]
    largest = torch.zeros_like(scales, dtype=x.dtype).index_reduce_(0, page, x.abs().amax(2), "amax")[touched]
    first = torch.full((scales.shape[0],), size, device=x.device).index_reduce_(0, page, off, "amin")[touched]
    before = torch.where((first == 0).unsqueeze(1), torch.zeros_like(largest, dtype=scales.dtype), scales[touched])
    after = torch.maximum(before, (largest / 127).to(scales.dtype))
    factor = before.double() / torch.where(after > 0, after, torch.ones_like(after)).double()
    again = torch.round(values[touched].double() * factor.unsqueeze(1).unsqueeze(3)).to(values.dtype)
    live = torch.arange(size, device=x.device).unsqueeze(0) < first.unsqueeze(1)
    values[touched] = torch.where(live.unsqueeze(2).unsqueeze(3), again, values[touched])
    scales[touched] = after
    s = scales[page].double()
    s = torch.where(s > 0, s, torch.ones_like(s))
    values[page, off] = torch.round(x / s.unsqueeze(2)).clamp(-127, 127).to(values.dtype)


def _plain_append(st, k, v, q, lengths, start, touched):
    case, cache = st["case"], st["cache"]
    seq, pos = _rows_of(k.shape[0], lengths, start)
    kd = k.double().view(k.shape[0], case["kv_heads"], case["dim"])
    vd = v.double().view_as(kd)
    if st["rope"] is not None:
        kd = _rotate(kd, pos, st["rope"], st["interleaved"])
    page, off = st["table"][seq, pos // case["page"]].long(), pos % case["page"]
    _plain_store(cache["k"], cache["ks"], kd, page, off, touched)
    _plain_store(cache["v"], cache["vs"], vd, page, off, touched)
    if q is None:
        return None
    qf = q.float().view(q.shape[0], case["heads"], case["dim"])
    if st["rope"] is not None:
        qf = _rotate(qf, pos, st["rope"], st["interleaved"])
    return qf.half().view_as(q)


def _plain_read(st, lengths, start, rows):
    case, cache = st["case"], st["cache"]
    seq, pos = _rows_of(rows, lengths, start)
    page, off = st["table"][seq, pos // case["page"]].long(), pos % case["page"]
    k = cache["k"][page, off].float() * cache["ks"][page].unsqueeze(2)
    v = cache["v"][page, off].float() * cache["vs"][page].unsqueeze(2)
    return k.half().flatten(1), v.half().flatten(1)


def _plain_attend(st):
    """All sequences as one batch, padded to the longest and to the most rows."""
    case, cache = st["case"], st["cache"]
    h, kv, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    n, most, g = case["batch"], st["most"], h // kv
    lengths, start = st["lengths"].long(), st["start_new"].long()
    table = st["table"].long().clamp_min(0)
    k = (cache["k"][table].float() * cache["ks"][table].unsqueeze(2).unsqueeze(4)).flatten(1, 2).transpose(1, 2).contiguous()
    v = (cache["v"][table].float() * cache["vs"][table].unsqueeze(2).unsqueeze(4)).flatten(1, 2).transpose(1, 2).contiguous()
    key = torch.arange(k.shape[2], device=DEV)
    count = start[1:] - start[:-1]
    slot = torch.arange(most, device=DEV)
    there = slot.unsqueeze(0) < count.unsqueeze(1)
    place = torch.where(there, start[:-1].unsqueeze(1) + slot, torch.zeros_like(slot))
    q = st["q"].float()[place].view(n, most, kv, g, d).permute(0, 2, 1, 3, 4).reshape(n, kv, most * g, d)
    score = torch.matmul(q, k.transpose(2, 3)) * (1 / math.sqrt(d))
    pos = (lengths - count).unsqueeze(1) + slot
    seen = (key < lengths.view(n, 1, 1)).expand(n, most, key.numel())
    if case["causal"]:
        seen = seen & (key <= pos.unsqueeze(2))
    if case["window"]:
        seen = seen & (key > (pos - case["window"]).unsqueeze(2))
    seen = seen.unsqueeze(2).expand(n, most, g, key.numel()).reshape(n, 1, most * g, key.numel())
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(3, keepdim=True)
    part = torch.where(seen, torch.exp(score - top), torch.zeros_like(score))
    out = torch.matmul(part, v) / part.sum(3, keepdim=True)
    out = out.view(n, kv, most, g, d).permute(0, 2, 1, 3, 4).reshape(n * most, h * d)
    seq = torch.searchsorted(start, torch.arange(st["q"].shape[0], device=DEV), right=True) - 1
    return out[seq * most + torch.arange(st["q"].shape[0], device=DEV) - start[seq]].half()


def run(st):
    case = st["case"]
    if case["op"] == "norm":
        if not own:
            return _plain_norm(st)
        import binary_rank_gemv_littlebitlinear_amd as lbm
        lbm.lb_norm(st["r"], x=st["x"], y=st["y"], out=st["out"], kind=case["kind"], weight=st["weight"], bias=st["bias"],
                    post=case["post"], post_weight=st["post_weight"], post_bias=st["post_bias"], gate=st["gate"],
                    scale=case["scale"], eps=1e-5)
        return {"x": st["x"], "r": st["out"]}
    if case["op"] == "append":
        if not own:
            q = _plain_append(st, st["k_new"], st["v_new"], st["q"], st["lengths"], st["start"], st["touched"])
            k, v = _plain_read(st, st["lengths"], st["start_back"], st["k_back"].shape[0])
            return {"q": q, "k": k, "v": v}
        st["cache"].append(st["k_new"], st["v_new"], st["lengths"], st["table"], start=st["start"], q=st["q"],
                           q_out=st["q_out"], rope=st["rope"], interleaved=st["interleaved"])
        st["cache"].read(st["k_back"], st["v_back"], st["lengths"], st["table"], start=st["start_back"])
        return {"q": st["q_out"], "k": st["k_back"], "v": st["v_back"]}
    if not own:
        return _plain_attend(st)
    st["cache"].attend(st["q"], st["out"], st["lengths"], st["table"], start=st["start"], max_length=st["longest"],
                       causal=case["causal"], window=case["window"])
    return st["out"]


# ------------------------------------------------------------------- exact
def _exact_norm(st, case):
    def standard(v, weight, bias):
        mean = v.sum(1, keepdim=True) / v.shape[1] if case["kind"] == "layer" else 0.0
        v = (v - mean) * torch.rsqrt(((v - mean) ** 2).sum(1, keepdim=True) / v.shape[1] + 1e-5)
        v = v if weight is None else v * weight.double()
        return v if bias is None else v + bias.double()

    r = st["y"].double()
    if case["post"]:
        r = standard(r, st["post_weight"], st["post_bias"])
    if st["gate"] is not None:
        r = st["gate"].double() * r
    if st["r"] is not None:
        r = r + st["r"].double() * case["scale"]
    return {"x": standard(r, st["weight"], st["bias"]), "r": r}


def _exact_turn(x, positions, case):
    """x [tokens, heads, dim]: pairs as complex numbers, times exp(i angle)."""
    rot = case["rot"]
    angle = torch.arange(rot // 2, device=DEV).double().mul(-2.0 / rot * math.log(10000.0)).exp()
    angle = positions.double().unsqueeze(1) * angle
    unit = torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    y = x.clone()
    even, odd = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * unit
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _exact_pages(old, new, page):
    """What a sequence's tokens [tokens, heads, dim] read as, page by page: those of the first call at the scale of
    their largest, rounded again where the second call brings a larger one."""
    both = torch.cat([old, new])
    out = torch.empty_like(both)
    n_old, n = old.shape[0], both.shape[0]
    full = n_old // page * page  # pages that the second call does not touch
    for lo, hi, at in ((0, full, full), (full, min(n, full + page), n_old), (full + page, n, 0)):
        if lo >= hi:
            continue
        pages = -(-(hi - lo) // page)
        x = torch.zeros((pages * page, *both.shape[1:]), dtype=torch.float64, device=DEV)
        x[: hi - lo] = both[lo:hi]
        x = x.view(pages, page, *both.shape[1:])
        step = x.abs().amax((1, 3), keepdim=True) / 127
        safe = torch.where(step > 0, step, 1.0)
        number = torch.round(x / safe)
        if lo < at < hi:  # the page that both calls write
            before = x[:, : at - lo].abs().amax((1, 3), keepdim=True) / 127
            kept = torch.round(x[:, : at - lo] / torch.where(before > 0, before, 1.0))
            number[:, : at - lo] = torch.round(kept * (before / safe))
        out[lo:hi] = (number * step).flatten(0, 1)[: hi - lo]
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st, case)
    lengths, new = _sequences(case)
    h, kv, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    turn = case["op"] == "append" and case["rot"] > 0
    at_old = at_new = 0
    found = {"q": [], "k": [], "v": []} if case["op"] == "append" else []
    for n, m in zip(lengths, new):
        o, w = slice(at_old, at_old + n - m), slice(at_new, at_new + m)
        at_old, at_new = at_old + n - m, at_new + m
        position = torch.arange(n, device=DEV)
        k, v = ([st[x + "_old"][o].double().view(-1, kv, d), st[x + "_new"][w].double().view(-1, kv, d)] for x in "kv")
        if turn:
            k = [_exact_turn(k[0], position[: n - m], case), _exact_turn(k[1], position[n - m:], case)]
        k, v = _exact_pages(*k, page), _exact_pages(*v, page)
        q = st["q"][w].double().view(m, h, d)
        if case["op"] == "append":
            first = (n - m) // page * page
            found["q"].append((_exact_turn(q, position[n - m:], case) if turn else q).flatten(1))
            found["k"].append(k[first:].flatten(1))
            found["v"].append(v[first:].flatten(1))
            continue
        mine = position[n - m:].unsqueeze(1)
        hidden = torch.zeros((m, n), dtype=torch.bool, device=DEV)
        if case["causal"]:
            hidden |= position > mine
        if case["window"]:
            hidden |= position <= mine - case["window"]
        out = torch.empty((m, h, d), dtype=torch.float64, device=DEV)
        for j in range(h):
            score = (q[:, j] @ k[:, j * kv // h].t().contiguous()) / math.sqrt(d)
            out[:, j] = torch.softmax(score.masked_fill(hidden, -math.inf), 1) @ v[:, j * kv // h].contiguous()
        found.append(out.flatten(1))
    if case["op"] == "append":
        return {name: torch.cat(x) for name, x in found.items()}
    return torch.cat(found)
