"""The decoder operators around the ternary projections, as measured cases: the
RMS norm with the residual's addition and 8-bit output, the append to an 8-bit
paged cache with rotary positions of several axes, and the attention over that
cache (single tokens, draft-verify batches, prompt chunks, sliding window with
sinks).

`run` computes each operator in elementary torch operations in 32 bits, or,
where `own` is true, through the calls of ternary_weight_linear_amd. `exact`
computes the same from the definitions in 64 bits.

The cache (the format both forms work on), pages of 64 tokens:
  k        int8  [pages, kv heads, 64, d]         slot t of a page holds one token
  v        int8  [pages, kv heads, d, 64]         token slot t at place V_PLACE[t]
  k_scale, v_scale  float32 [pages, kv heads]     value = code * scale
"""
import math

import torch

own = False

PAGE = 64
EPS = 1e-6


def v_place(t):
    """Place of token slot t (0..63) in a row of v: slots 4g..4g+3 of the four
    16-token tiles lie next to each other, tile by tile."""
    return 16 * ((t % 16) // 4) + 4 * (t // 16) + t % 4


# ------------------------------------------------------------------ cases
#
# Head layouts: 40 query heads of 128 (the 5120-wide projections of this
# repository's layers) over 8 kv heads; 64 and 256 wide heads as further
# generic layouts. Token counts and chunk sizes are those of the repository's
# rungs (1, 4, 17, 508, 2048) and prefill chunk (1024), or generic.


def _norm(name, T, K, x, r, out):
    return {"name": name, "op": "norm", "T": T, "K": K, "x": x, "r": r, "out": out}


def _append(name, seqs, q, ctx, hq, hkv, d, rot, axes, src):
    return {"name": name, "op": "append", "seqs": seqs, "q": q, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d,
            "rot": rot, "axes": axes, "src": src}


def _attn(name, seqs, q, ctx, hq, hkv, d, window=0, sinks=0):
    return {"name": name, "op": "attn", "seqs": seqs, "q": q, "ctx": ctx, "hq": hq, "hkv": hkv, "d": d,
            "window": window, "sinks": sinks}


def listed():
    return [
        # one decoded token between two projections: nothing but latency
        _norm("norm one token", 1, 5120, "f32", "f32", "s8"),
        # a short prompt with an odd number of tokens, bf16 stream
        _norm("norm 509 tokens bf16", 509, 5120, "bf16", "bf16", "s8"),
        # a prefill step on the projections' 32-bit outputs
        _norm("norm prefill 2048", 2048, 5120, "f32", "f32", "s8"),
        # one decode step of a batch: every sequence adds one token to a page that holds some
        _append("append decode 32", 32, 1, 4000, 40, 8, 128, 128, 3, "f32"),
        # a prompt chunk with images in it, starting inside a page
        _append("append prompt 2048", 1, 2048, 3001, 40, 8, 128, 128, 3, "f32"),
        # the first tokens of one conversation: the smallest attention
        _attn("attn one short", 1, 1, 17, 40, 8, 128),
        # a decode step of a full batch, lengths spread over 1:8
        _attn("attn decode 32", 32, 1, 8192, 40, 8, 128),
        # one conversation with a long context
        _attn("attn decode long", 1, 1, 131072, 40, 8, 128),
        # draft-verify: four tokens a sequence
        _attn("attn verify 16x4", 16, 4, 4095, 40, 8, 128),
        # a prefill chunk on top of a context
        _attn("attn prompt 1024", 1, 1024, 8192, 40, 8, 128),
        # decode with a sliding window and sinks on long contexts, 64 wide heads
        _attn("attn window decode 64", 64, 1, 32768, 64, 8, 64, 4096, 4),
        # prompt chunks of several sequences with a window, 256 wide heads
        _attn("attn window prompt 3x508", 3, 508, 6001, 24, 4, 256, 1024, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "append", "attn", "attn", "attn"])
    if op == "norm":
        c = _norm("", _log(rng, 1, 2048), 64 * _log(rng, 4, 272), rng.choice(["f32", "bf16"]),
                  rng.choice(["f32", "bf16", "none"]), rng.choice(["s8", "s8", "bf16"]))
        while c["T"] * c["K"] > 2048 * 5120:
            c["T"] = (c["T"] + 1) // 2
    elif op == "append":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 8])
        d = rng.choice([64, 128, 128, 256])
        seqs, q = (_log(rng, 1, 64), 1) if rng.random() < 0.4 else (rng.randint(1, 4), _log(rng, 2, 1024))
        while seqs * q * (hq + 2 * hkv) * d > 2048 * 56 * 128:
            q = (q + 1) // 2
        c = _append("", seqs, q, q + _log(rng, 1, 4000), hq, hkv, d, rng.choice([d, d // 2]), rng.choice([1, 3]),
                    rng.choice(["f32", "bf16"]))
    else:
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 6, 8])
        d = rng.choice([64, 128, 128, 256])
        kind = rng.choice(["decode", "verify", "prompt"])
        if kind == "decode":
            seqs, q, ctx = _log(rng, 1, 64), 1, _log(rng, 1, 65536)
        elif kind == "verify":
            seqs, q, ctx = _log(rng, 1, 32), rng.randint(2, 8), _log(rng, 8, 16384)
        else:
            seqs, q = rng.randint(1, 4), _log(rng, 9, 1024)
            ctx = q + _log(rng, 1, 8192)
        while seqs * ctx * 2 * hkv * d > 131072 * 2048:
            ctx = max(q, ctx // 2)
            seqs = seqs if ctx > 4096 else (seqs + 1) // 2
        while seqs * q * ctx * hq * d > 1024 * 8192 * 40 * 128:
            q = (q + 1) // 2
        window, sinks = (_log(rng, 16, 4096), rng.choice([0, 1, 4, 64])) if rng.random() < 0.35 else (0, 0)
        c = _attn("", seqs, q, max(ctx, q), hq, hkv, d, window, sinks)
    del c["name"]
    return c


# ----------------------------------------------------------------- shapes


def _lengths(c):
    """Tokens in the cache of each sequence, this call's among them: spread
    from ctx down to about ctx / 8, never less than the call's own tokens."""
    return [max(c["q"], c["ctx"] - i * c["ctx"] * 7 // (8 * c["seqs"])) for i in range(c["seqs"])]


def _first_read(c):
    """First token of the pages that an append touches, for each sequence."""
    return [(n - c["q"]) // PAGE * PAGE for n in _lengths(c)]


def _seen(c, n):
    """(tokens that some query sees, pairs of query and visible key) of a sequence of n tokens."""
    w, s, tokens, pairs = c["window"], c["sinks"], 0, 0
    for i in range(n - c["q"], n):
        first = max(0, i - w + 1) if w else 0
        pairs += i + 1 - first + min(s, first)
    first = max(0, n - c["q"] - w + 1) if w else 0
    tokens = n - first + min(s, first)
    return tokens, pairs


_BYTES = {"f32": 4, "bf16": 2, "none": 0}


def work(c):
    if c["op"] == "norm":
        e = c["T"] * c["K"]
        out = 1 if c["out"] == "s8" else 2
        return {"bytes": e * (_BYTES[c["x"]] + 2 * _BYTES[c["r"]] + out) + 4 * c["K"] + 4 * c["T"], "flops": 8 * e}
    rows = c["seqs"] * c["q"]
    if c["op"] == "append":
        kept = sum(n - c["q"] - f for n, f in zip(_lengths(c), _first_read(c)))
        src = rows * (c["hq"] + 2 * c["hkv"]) * c["d"] * _BYTES[c["src"]]
        got = rows * c["hq"] * c["d"] * 2 + rows * 2 * c["hkv"] * c["d"]
        back = (kept + rows) * 2 * c["hkv"] * c["d"] * 3  # the touched pages' values: codes read, bf16 written
        return {"bytes": src + got + back + rows * c["rot"] * 4, "flops": 6 * rows * (c["hq"] + 2 * c["hkv"]) * c["d"]}
    seen = [_seen(c, n) for n in _lengths(c)]
    tokens, pairs = sum(t for t, _ in seen), sum(p for _, p in seen)
    return {"bytes": tokens * 2 * c["hkv"] * c["d"] + 4 * rows * c["hq"] * c["d"] + tokens // PAGE * 8 * c["hkv"],
            "flops": 4 * pairs * c["hq"] * c["d"]}


# ---------------------------------------------------------------- inputs

_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _outliers(g, n):
    """Channel magnitudes: 1 % of the channels are 20 times larger."""
    return torch.where(torch.rand(n, generator=g, device="cuda") < 0.01, 20.0, 1.0)


def _to_codes(x):
    """Codes and scales of pages x [pages, heads, tokens, d]."""
    s = x.abs().amax((2, 3)) / 127
    return torch.round(x / s[:, :, None, None]).clamp(-127, 127).to(torch.int8), s


def _cache(c, g):
    """A cache with every sequence's tokens in pages of random order, and its table."""
    lens = _lengths(c)
    need = [(n + PAGE - 1) // PAGE for n in lens]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    k = torch.empty((pages, c["hkv"], PAGE, c["d"]), dtype=torch.int8, device="cuda")
    v = torch.empty((pages, c["hkv"], c["d"], PAGE), dtype=torch.int8, device="cuda")
    ks = torch.empty((pages, c["hkv"]), device="cuda")
    vs = torch.empty((pages, c["hkv"]), device="cuda")
    place = torch.tensor([v_place(t) for t in range(PAGE)], device="cuda")
    size = 0.5 + torch.rand((c["hkv"], 1, c["d"]), generator=g, device="cuda")
    for p in range(0, pages, 256):
        n = min(256, pages - p)
        k[p:p + n], ks[p:p + n] = _to_codes(_normal(g, n, c["hkv"], PAGE, c["d"]) * size)
        codes, vs[p:p + n] = _to_codes(_normal(g, n, c["hkv"], PAGE, c["d"]) * (0.2 + torch.rand((n, 1, 1, 1), generator=g, device="cuda")))
        v[p:p + n, :, :, place] = codes.transpose(2, 3)
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs, "table": table, "place": place,
            "kv_len": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "q_begin": torch.arange(c["seqs"] + 1, dtype=torch.int32, device="cuda") * c["q"]}


def _positions(c, g):
    """Rotary positions [axes, tokens] of the new tokens: text, with an image of
    rows x columns in every prompt that is long enough for one."""
    out = torch.empty((c["seqs"], c["axes"], c["q"]), dtype=torch.int64, device="cuda")
    j = torch.arange(c["q"], device="cuda")
    for i, n in enumerate(_lengths(c)):
        start = n - c["q"]
        out[i] = start + j
        if c["axes"] == 3 and c["q"] >= 64:
            a, cols = c["q"] // 4, max(2, int(math.sqrt(c["q"] // 2)))
            b = a + c["q"] // 2
            m = j[a:b] - a
            out[i, 0, a:b] = start + a
            out[i, 1, a:b] = start + a + m // cols
            out[i, 2, a:b] = start + a + m % cols
    return out.permute(1, 0, 2).reshape(c["axes"], -1).to(torch.int32).contiguous()


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "norm":
        s = {"x": (_normal(g, c["T"], c["K"]) * _outliers(g, c["K"])).to(_TYPE[c["x"]]),
             "w": 1 + 0.1 * _normal(g, c["K"]),
             "r": None if c["r"] == "none" else (3 * _normal(g, c["T"], c["K"]) * _outliers(g, c["K"])).to(_TYPE[c["r"]])}
    elif c["op"] == "append":
        s = _cache(c, g)
        rows, width = c["seqs"] * c["q"], (c["hq"] + 2 * c["hkv"]) * c["d"]
        # the q/k/v projection's output, in one matrix
        s["qkv"] = (_normal(g, rows, width) * _outliers(g, width)).to(_TYPE[c["src"]])
        s["positions"] = _positions(c, g)
        half, most = c["rot"] // 2, int(max(_lengths(c))) + 64
        f = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        a = torch.arange(most, dtype=torch.float64, device="cuda")[:, None] * f
        s["rope"] = torch.stack((a.cos(), a.sin()), -1).float().contiguous()  # [positions, pairs, 2]
        # axis of each pair: one quarter time, then height and width in turn
        i = torch.arange(half, device="cuda")
        s["axis"] = (torch.where(i < half // 4, 0, 1 + (i - half // 4) % 2) if c["axes"] == 3 else 0 * i).to(torch.uint8)
        first = _first_read(c)
        n = [0]
        for x, f0 in zip(_lengths(c), first):
            n.append(n[-1] + x - f0)
        s["read_begin"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        s["read_rows"], s["read_most"] = n[-1], max(b - a for a, b in zip(n, n[1:]))
    else:
        s = _cache(c, g)
        rows = c["seqs"] * c["q"]
        s["q"] = (1.5 * _normal(g, rows, c["hq"], c["d"])).to(torch.bfloat16)
    s["case"] = c
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps from call to call: the cache's and the batches' handles, the workspace."""
    import ternary_weight_linear_amd as tl
    s["tl"], c = tl, s["case"]
    if c["op"] == "norm":
        return
    most = max(_lengths(c))
    s["cache"] = tl.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    s["batch"] = tl.KVBatch(s["q_begin"], s["kv_len"], s["table"], max_q=c["q"], max_kv=most)
    if c["op"] == "append":
        s["reads"] = tl.KVBatch(s["read_begin"], s["kv_len"], s["table"], max_q=s["read_most"], max_kv=most)
        s["turn"] = tl.Rope(s["rope"], s["axis"])
    else:
        s["workspace"] = tl.kv_attn_workspace(s["cache"], s["batch"], c["seqs"] * c["q"], c["hq"], c["window"], c["sinks"])


# ----------------------------------------------------------- the operators


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_norm(state) if op == "norm" else _own_append(state) if op == "append" else _own_attn(state)
    return _plain_norm(state) if op == "norm" else _plain_append(state) if op == "append" else _plain_attn(state)


def _own_norm(s):
    tl, c, r = s["tl"], s["case"], s["r"]
    out = None if r is None else torch.empty_like(r)  # not in place: every pass starts from the same stream
    if c["out"] == "bf16":
        return {"y": tl.rmsnorm(s["x"], s["w"], EPS, residual=r, residual_out=out), "residual": out}
    q, scale = tl.rmsnorm_s8(s["x"], s["w"], EPS, residual=r, residual_out=out)
    return {"values": torch.mul(q, scale[:, None], out=torch.empty_like(q, dtype=torch.bfloat16)), "residual": out}


def _plain_norm(s):
    r, c = s["r"], s["case"]
    h = s["x"].float()
    if r is not None:
        r = (h + r.float()).to(r.dtype)
        h = r.float()
    rho = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    v = h * s["w"]
    if c["out"] == "bf16":
        return {"y": (v * rho).to(torch.bfloat16), "residual": r}
    scale = v.abs().amax(1, keepdim=True) / 127
    codes = torch.round(v / scale).clamp(-127, 127)
    return {"values": (codes * (rho * scale)).to(torch.bfloat16), "residual": r}


def _split(s):
    c = s["case"]
    a, b = c["hq"] * c["d"], (c["hq"] + c["hkv"]) * c["d"]
    x = s["qkv"]
    return (x[:, :a].unflatten(1, (c["hq"], c["d"])), x[:, a:b].unflatten(1, (c["hkv"], c["d"])),
            x[:, b:].unflatten(1, (c["hkv"], c["d"])))


def _own_append(s):
    tl = s["tl"]
    q, k, v = _split(s)
    q = tl.kv_append(s["cache"], s["batch"], k, v, q=q, rope=s["turn"], positions=s["positions"])
    k, v = tl.kv_read(s["cache"], s["reads"], s["read_rows"])
    return {"q": q, "k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _turned(s, x):
    """x [tokens, heads, d] in 32 bits, turned by its tokens' positions."""
    half = s["case"]["rot"] // 2
    i = torch.arange(half, device=x.device)
    cs = s["rope"][s["positions"].long()[s["axis"].long()], i[:, None]].transpose(0, 1)[:, None]  # [tokens, 1, pairs, 2]
    a, b = x[..., :half], x[..., half:2 * half]
    return torch.cat((a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1], x[..., 2 * half:]), -1)


def _tokens(s, begin, count):
    """(sequence, position) of each of `count` rows: the last tokens of every sequence."""
    row = torch.arange(count, dtype=torch.int32, device=begin.device)
    seq = torch.searchsorted(begin, row, right=True) - 1
    return seq, s["kv_len"].long()[seq] - begin.long()[seq + 1] + row


def _plain_append(s):
    c = s["case"]
    q, k, v = (x.float() for x in _split(s))
    q, k = _turned(s, q).to(torch.bfloat16), _turned(s, k)
    begin, table = s["q_begin"], s["table"].long()
    seq, pos = _tokens(s, begin, q.shape[0])
    page, slot = table[seq, pos // PAGE], pos % PAGE
    start = s["kv_len"].long() - begin.diff()
    inside = start % PAGE > 0  # sequences whose first touched page holds tokens already
    kept = table.gather(1, (start // PAGE)[:, None])[:, 0].clamp_min(0)
    place = s["place"]
    for x, codes, scale in ((k, s["k"], s["k_scale"]), (v, s["v"], s["v_scale"])):
        top = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(2), "amax") / 127
        new = scale.clone()
        new[page] = top[page]
        old = scale[kept]
        new[kept] = torch.where(inside[:, None], torch.maximum(old, top[kept]), new[kept])
        scale.copy_(new)
        keep = torch.round(codes[kept].float() * old[:, :, None, None] / new[kept][:, :, None, None])
        codes[kept] = torch.where(inside[:, None, None, None], keep, codes[kept].float()).clamp(-127, 127).to(torch.int8)
        fresh = torch.round(x / new[page][:, :, None]).clamp(-127, 127).to(torch.int8)
        if codes is s["k"]:
            codes[page, :, slot] = fresh
        else:
            codes[page, :, :, place[slot]] = fresh
    seq, pos = _tokens(s, s["read_begin"], s["read_rows"])
    page, slot = table[seq, pos // PAGE], pos % PAGE
    k = s["k"][page, :, slot].float() * s["k_scale"][page][:, :, None]
    v = s["v"][page, :, :, place[slot]].float() * s["v_scale"][page][:, :, None]
    return {"q": q, "k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _own_attn(s):
    c = s["case"]
    return s["tl"].kv_attn(s["q"], s["cache"], s["batch"], c["d"] ** -0.5, window=c["window"], sinks=c["sinks"],
                           workspace=s["workspace"])


def _visible(c, kv_len, keys, device):
    """[seqs, queries, keys]: whether the query sees the key."""
    i = kv_len.long()[:, None, None] - c["q"] + torch.arange(c["q"], device=device)[None, :, None]
    j = torch.arange(keys, device=device)[None, None, :]
    see = j <= i
    return see & ((j > i - c["window"]) | (j < c["sinks"])) if c["window"] else see


def _plain_attn(s):
    c = s["case"]
    n, hkv, d = c["seqs"], c["hkv"], c["d"]
    table = s["table"][:, :-1].long().clamp_min(0)
    keys = table.shape[1] * PAGE
    # [seqs, kv heads, keys, d]
    k = (s["k"][table].float() * s["k_scale"][table][..., None, None]).transpose(1, 2).reshape(n, hkv, keys, d)
    v = (s["v"][table][..., s["place"]].float() * s["v_scale"][table][..., None, None]).transpose(3, 4)
    v = v.transpose(1, 2).reshape(n, hkv, keys, d)
    q = s["q"].float().view(n, c["q"], hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5).view(n, hkv, -1, c["q"], keys)
    see = _visible(c, s["kv_len"], keys, x.device)[:, None, None]
    x.masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, hkv, -1, keys), v).view(n, hkv, -1, c["q"], d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(n * c["q"], c["hq"], d).to(torch.bfloat16)


# ------------------------------------------------------- in 64 bits, apart


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    return _exact_append(s) if case["op"] == "append" else _exact_attn(s)


def _exact_norm(s):
    h = s["x"].double()
    r = None
    if s["r"] is not None:
        h = h + s["r"].double()
        r = h
        h = h.to(s["r"].dtype).double()  # the norm is that of the stream as it is stored
    y = h * torch.rsqrt(h.pow(2).mean(1, keepdim=True) + EPS) * s["w"].double()
    if s["case"]["out"] == "bf16":
        return {"y": y, "residual": r}
    step = y.abs().amax(1, keepdim=True) / 127
    return {"values": torch.round(y / step).clamp(-127, 127) * step, "residual": r}


def _exact_append(s):
    c = s["case"]
    x = s["qkv"].double().view(c["seqs"], c["q"], -1, c["d"])
    half = c["rot"] // 2
    ang = torch.stack([s["rope"][s["positions"][a].long()].double() for a in range(c["axes"])])  # [axes, tokens, pairs, 2]
    axis = s["axis"].long()
    cs = torch.stack([ang[int(axis[i]), :, i] for i in range(half)], 1).view(c["seqs"], c["q"], 1, half, 2)
    heads = c["hq"] + c["hkv"]
    turn = x[:, :, :heads].clone()
    turn[..., :half] = x[:, :, :heads, :half] * cs[..., 0] - x[:, :, :heads, half:2 * half] * cs[..., 1]
    turn[..., half:2 * half] = x[:, :, :heads, half:2 * half] * cs[..., 0] + x[:, :, :heads, :half] * cs[..., 1]
    back = [[], []]
    scales = [s["k_scale"].double().clone(), s["v_scale"].double().clone()]
    table = s["table"].long().cpu()
    place = s["place"]
    for b, n in enumerate(_lengths(c)):
        start = n - c["q"]
        for p in range(start // PAGE, (n + PAGE - 1) // PAGE):
            lo, hi, page = max(start, p * PAGE), min(n, (p + 1) * PAGE), int(table[b, p])
            for which, codes in ((0, s["k"][page].double()), (1, s["v"][page][:, :, place].transpose(1, 2).double())):
                new = (turn[b, lo - start:hi - start, c["hq"]:] if which == 0 else x[b, lo - start:hi - start, heads:]).transpose(0, 1)
                step = new.abs().amax((1, 2)) / 127
                held = codes[:, :lo - p * PAGE]
                if lo > p * PAGE:
                    old = scales[which][page].clone()
                    step = torch.maximum(step, old)
                    held = torch.round(held * old[:, None, None] / step[:, None, None])
                held = torch.cat((held, torch.round(new / step[:, None, None]).clamp(-127, 127)), 1)
                scales[which][page] = step
                back[which].append((held * step[:, None, None]).transpose(0, 1))
    return {"q": turn[:, :, :c["hq"]].reshape(-1, c["hq"], c["d"]), "k": torch.cat(back[0]), "v": torch.cat(back[1]),
            "k_scale": scales[0], "v_scale": scales[1]}


def _exact_attn(s):
    c = s["case"]
    group = c["hq"] // c["hkv"]
    out = torch.zeros((c["seqs"] * c["q"], c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    table = s["table"].long()
    for b, n in enumerate(_lengths(c)):
        pages = table[b, :(n + PAGE - 1) // PAGE]
        at = torch.arange(n - c["q"], n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None]
        hide = key > at
        if c["window"]:
            hide = hide | ((key <= at - c["window"]) & (key >= c["sinks"]))
        for h in range(c["hkv"]):
            k = (s["k"][pages, h].double() * s["k_scale"][pages, h, None, None].double()).reshape(-1, c["d"])[:n]
            v = s["v"][pages, h][:, :, s["place"]].transpose(1, 2).double() * s["v_scale"][pages, h, None, None].double()
            v = v.reshape(-1, c["d"])[:n]
            for g in range(h * group, (h + 1) * group):
                x = (s["q"][b * c["q"]:(b + 1) * c["q"], g].double() @ k.T) / math.sqrt(c["d"])
                out[b * c["q"]:(b + 1) * c["q"], g] = torch.softmax(x.masked_fill(hide, -math.inf), 1) @ v
    return out
