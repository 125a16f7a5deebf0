"""The operators of a decoder's recurrent block around the ternary projections,
as measured cases: the short causal convolution with its state, the selective
state space scan (single tokens, drafts, prompts), the gated norm in front of
the output projection, and the norm behind a block with residual scale, sum and
the next block's norm.

`run` computes each operator in elementary torch operations in 32 bits, or,
where `own` is true, through the calls of ternary_weight_linear_amd. `exact`
computes the same from the definitions in 64 bits.

Sequences are ragged: rows begin[s] .. begin[s + 1] - 1 of the token matrices
belong to sequence s, which reads the state slot src[s] and leaves its state in
slot dst[s]. The passes read and write different slots, as a program does that
may take a draft's tokens back, so every pass starts from the same state.
  convolution state  [slots, width - 1, channels], the last inputs, oldest first
  scan state         float32 [slots, heads, n, p]
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases
#
# The block of a 5120-wide decoder: 10240 inner channels in 160 heads of 64,
# state width 128, 8 groups that share B and C; the input projection gives z
# (10240), x, B and C (12288, through the convolution) and dt (160). Further
# head layouts are generic. Token counts and chunk sizes are those of the
# repository's rungs (1, 4, 17, 508, 2048) and prefill chunk (1024), or generic.


def _conv(name, seqs, q, ch, width, x, act=True, bias=True):
    return {"name": name, "op": "conv", "seqs": seqs, "q": q, "ch": ch, "width": width, "x": x, "act": act, "bias": bias}


def _scan(name, seqs, q, heads, p, n, groups, fresh=False, dt="f32", softplus=True, skip=True):
    return {"name": name, "op": "scan", "seqs": seqs, "q": q, "heads": heads, "p": p, "n": n, "groups": groups,
            "fresh": fresh, "dt": dt, "softplus": softplus, "skip": skip}


def _gated(name, T, K, group, x, z, out, first=True):
    return {"name": name, "op": "gated", "T": T, "K": K, "group": group, "x": x, "z": z, "out": out, "first": first}


def _post(name, T, K, x, r, out, gate="none"):
    return {"name": name, "op": "post", "T": T, "K": K, "x": x, "r": r, "out": out, "gate": gate}


def listed():
    return [
        # a decode step of a full batch, on bf16 rows
        _conv("conv decode 32", 32, 1, 12288, 4, "bf16"),
        # a prefill step on the projection's 32-bit output
        _conv("conv prompt 2048", 1, 2048, 12288, 4, "f32"),
        # one decoded token of one conversation: nothing but latency
        _scan("scan one token", 1, 1, 160, 64, 128, 8),
        # a decode step of a full batch
        _scan("scan decode 32", 32, 1, 160, 64, 128, 8),
        # draft-verify: four tokens a sequence, the state before them kept
        _scan("scan verify 16x4", 16, 4, 160, 64, 128, 8),
        # a prefill step that goes on from a state
        _scan("scan prompt 2048", 1, 2048, 160, 64, 128, 8),
        # new prompts of several conversations, 128 wide heads, one group
        _scan("scan prompts 3x509", 3, 509, 40, 128, 64, 1, fresh=True, dt="bf16"),
        # a long prompt with few heads, as one of several that share a model would hold them
        _scan("scan long 8192", 1, 8192, 20, 64, 128, 1),
        # in front of the output projection's 8-bit rung in a prefill step
        _gated("gated norm prefill 2048", 2048, 10240, 1280, "bf16", "f32", "s8"),
        # norms of single heads, gated after the norm
        _gated("gated norm heads 509", 509, 5120, 128, "bf16", "bf16", "bf16", first=False),
        # behind the output projection in a decode step of a small batch
        _post("post norm 17 tokens", 17, 5120, "f32", "f32", "bf16"),
        # behind the output projection in a prefill step, in front of an 8-bit projection
        _post("post norm prefill 2048", 2048, 5120, "f32", "f32", "s8", gate="channels"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "scan", "gated", "post"])
    if op == "conv":
        seqs, q = (_log(rng, 1, 64), rng.choice([1, 1, 2, 4])) if rng.random() < 0.4 else (rng.randint(1, 4), _log(rng, 9, 2048))
        c = _conv("", seqs, q, 8 * _log(rng, 32, 1536), rng.choice([2, 3, 4, 4]), rng.choice(["f32", "bf16"]),
                  rng.random() < 0.8, rng.random() < 0.7)
        while c["seqs"] * c["q"] * c["ch"] > 2048 * 12288:
            c["q"] = (c["q"] + 1) // 2
    elif op == "scan":
        groups = rng.choice([1, 1, 2, 4, 8])
        heads = groups * rng.choice([1, 2, 3, 4, 5, 10, 20])
        p, n = rng.choice([32, 64, 64, 128]), rng.choice([64, 128, 128, 256])
        kind = rng.choice(["decode", "verify", "prompt", "prompt"])
        if kind == "decode":
            seqs, q = _log(rng, 1, 64), 1
        elif kind == "verify":
            seqs, q = _log(rng, 1, 32), rng.randint(2, 8)
        else:
            seqs, q = rng.randint(1, 4), _log(rng, 9, 4096)
        while seqs * heads * p * n > 32 * 160 * 64 * 128:
            seqs = (seqs + 1) // 2
        while seqs * q * heads * p * n > 2048 * 160 * 64 * 128:
            q = (q + 1) // 2
        c = _scan("", seqs, q, heads, p, n, groups, rng.random() < 0.3, rng.choice(["f32", "f32", "bf16"]),
                  rng.random() < 0.85, rng.random() < 0.8)
    elif op == "gated":
        group = 64 * _log(rng, 1, 40)
        c = _gated("", _log(rng, 1, 2048), group * rng.randint(1, max(1, min(8, 16384 // group))), group,
                   rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]), rng.choice(["s8", "bf16"]), rng.random() < 0.6)
        while c["T"] * c["K"] > 2048 * 10240:
            c["T"] = (c["T"] + 1) // 2
    else:
        c = _post("", _log(rng, 1, 2048), 64 * _log(rng, 4, 272), rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"]),
                  rng.choice(["s8", "bf16"]), rng.choice(["none", "channels", "tokens"]))
        while c["T"] * c["K"] > 2048 * 5120:
            c["T"] = (c["T"] + 1) // 2
    del c["name"]
    return c


def _lengths(c):
    """Tokens of each sequence in this call: from q down to about q / 2."""
    return [c["q"] - i * c["q"] // (2 * c["seqs"]) for i in range(c["seqs"])]


_BYTES = {"f32": 4, "bf16": 2, "s8": 1}


def work(c):
    if c["op"] in ("gated", "post"):
        e = c["T"] * c["K"]
        if c["op"] == "gated":
            return {"bytes": e * (_BYTES[c["x"]] + _BYTES[c["z"]] + _BYTES[c["out"]]) + 4 * c["K"], "flops": 12 * e}
        gate = {"none": 0, "channels": 4 * c["K"], "tokens": 4 * e}[c["gate"]]
        return {"bytes": e * (_BYTES[c["x"]] + 2 * _BYTES[c["r"]] + _BYTES[c["out"]]) + 8 * c["K"] + gate, "flops": 12 * e}
    rows = sum(_lengths(c))
    if c["op"] == "conv":
        state = 2 * c["seqs"] * (c["width"] - 1) * c["ch"] * _BYTES[c["x"]]
        return {"bytes": rows * c["ch"] * (_BYTES[c["x"]] + 2) + state + 4 * c["ch"] * (c["width"] + 1),
                "flops": rows * c["ch"] * (2 * c["width"] + 4)}
    state = c["seqs"] * c["heads"] * c["n"] * c["p"] * 4 * (1 if c["fresh"] else 2)
    token = 4 * c["heads"] * c["p"] + 4 * c["groups"] * c["n"] + c["heads"] * _BYTES[c["dt"]]
    return {"bytes": rows * token + state, "flops": 5 * rows * c["heads"] * c["p"] * c["n"]}


# ---------------------------------------------------------------- inputs

_TYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _outliers(g, n):
    """Channel magnitudes: 1 % of the channels are 20 times larger."""
    return torch.where(_uniform(g, n) < 0.01, 20.0, 1.0)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "gated":
        s["x"] = (_normal(g, c["T"], c["K"]) * _outliers(g, c["K"])).to(_TYPE[c["x"]])
        # z is a slice of the input projection's rows
        s["z"] = _normal(g, c["T"], c["K"] + 256).to(_TYPE[c["z"]])[:, :c["K"]]
        s["w"] = 1 + 0.1 * _normal(g, c["K"])
    elif c["op"] == "post":
        s["x"] = (_normal(g, c["T"], c["K"]) * _outliers(g, c["K"])).to(_TYPE[c["x"]])
        s["r"] = (3 * _normal(g, c["T"], c["K"]) * _outliers(g, c["K"])).to(_TYPE[c["r"]])
        s["w_post"], s["w"] = 1 + 0.1 * _normal(g, c["K"]), 1 + 0.1 * _normal(g, c["K"])
        s["scale"] = 0.22
        s["gate"] = None
        if c["gate"] == "channels":
            s["gate"] = 1 + 0.1 * _normal(g, c["K"])
        elif c["gate"] == "tokens":
            s["gate"] = _normal(g, c["T"], c["K"])
    else:
        lens = _lengths(c)
        begin = [0]
        for n in lens:
            begin.append(begin[-1] + n)
        rows, slots = begin[-1], 2 * c["seqs"] + 1
        order = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
        s["begin"] = torch.tensor(begin, dtype=torch.int32, device="cuda")
        s["src"], s["dst"] = order[:c["seqs"]].contiguous(), order[c["seqs"]:2 * c["seqs"]].contiguous()
        if c["op"] == "conv":
            # the convolution's columns of the input projection's rows
            wide = _normal(g, rows, c["ch"] + 512) * _outliers(g, c["ch"] + 512)
            s["x"] = wide.to(_TYPE[c["x"]])[:, 256:256 + c["ch"]]
            s["w"] = _normal(g, c["ch"], c["width"]) / math.sqrt(c["width"])
            s["bias"] = 0.1 * _normal(g, c["ch"]) if c["bias"] else None
            s["state"] = _normal(g, slots, c["width"] - 1, c["ch"]).to(_TYPE[c["x"]])
        else:
            inner, shared = c["heads"] * c["p"], c["groups"] * c["n"]
            # x, B and C as the convolution leaves them, in one matrix
            s["xbc"] = torch.nn.functional.silu(_normal(g, rows, inner + 2 * shared)).to(torch.bfloat16)
            first = torch.exp(_uniform(g, c["heads"]) * math.log(100) + math.log(1e-3))  # steps from 1/1000 to 1/10
            s["a"] = -(1 + 15 * _uniform(g, c["heads"]))
            s["d"] = 1 + 0.1 * _normal(g, c["heads"]) if c["skip"] else None
            dt = 0.5 * _normal(g, rows, c["heads"] + 32)[:, :c["heads"]]
            if c["softplus"]:
                s["dt_bias"] = first + torch.log(-torch.expm1(-first))
                s["dt"] = dt.to(_TYPE[c["dt"]])
            else:
                s["dt_bias"] = None
                s["dt"] = (first * torch.exp(dt)).to(_TYPE[c["dt"]])
            s["state"] = 0.02 * _normal(g, slots, c["heads"], c["n"], c["p"])  # about as large as such inputs leave it
            if c["fresh"]:
                s["src"] = torch.full_like(s["src"], -1)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program keeps from call to call: the batch's handle, the workspace."""
    import ternary_weight_linear_amd as tl
    s["tl"], c = tl, s["case"]
    if c["op"] in ("gated", "post"):
        return
    s["batch"] = tl.StateBatch(s["begin"], s["src"], s["dst"], max_q=c["q"])
    if c["op"] == "scan":
        s["workspace"] = tl.scan_workspace(s["batch"], s["xbc"].shape[0], c["heads"], c["p"], c["groups"], c["n"])


# ----------------------------------------------------------- the operators


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _own_conv, "scan": _own_scan, "gated": _own_gated, "post": _own_post}[op](state)
    return {"conv": _plain_conv, "scan": _plain_scan, "gated": _plain_gated, "post": _plain_post}[op](state)


def _silu(x):
    return x / (1 + torch.exp(-x))


def _own_conv(s):
    y = s["tl"].causal_conv(s["x"], s["w"], s["state"], s["batch"], bias=s["bias"],
                            activation="silu" if s["case"]["act"] else None)
    return {"y": y, "state": s["state"]}


def _plain_conv(s):
    c, x, begin = s["case"], s["x"].float(), s["begin"].long()
    w, k, rows = s["w"], c["width"], x.shape[0]
    row = torch.arange(rows, device=x.device)
    seq = torch.searchsorted(begin, row, right=True) - 1
    inputs = torch.cat((x, s["state"][s["src"].long()].flatten(0, 1).float()))  # the call's rows, then the states'

    def place(seq, at):
        """Rows of `inputs` that hold the sequences' inputs number `at` of this call, those before it negative."""
        return torch.where(at >= 0, begin[seq] + at, rows + (k - 1) * (seq + 1) + at)

    sums = sum(inputs[place(seq, row - begin[seq] + j - (k - 1))] * w[:, j] for j in range(k))
    if s["bias"] is not None:
        sums = sums + s["bias"]
    each = torch.arange(c["seqs"], device=x.device)[:, None]
    last = place(each, begin.diff()[:, None] + torch.arange(1 - k, 0, device=x.device))
    s["state"][s["dst"].long()] = inputs[last].to(s["state"].dtype)
    return {"y": (_silu(sums) if c["act"] else sums).to(torch.bfloat16), "state": s["state"]}


def _parts(s):
    """x [rows, heads, p], B and C [rows, groups, n] of the convolution's output."""
    c, m = s["case"], s["xbc"]
    inner, shared = c["heads"] * c["p"], c["groups"] * c["n"]
    return (m[:, :inner].unflatten(1, (c["heads"], c["p"])), m[:, inner:inner + shared].unflatten(1, (c["groups"], c["n"])),
            m[:, inner + shared:].unflatten(1, (c["groups"], c["n"])))


def _own_scan(s):
    x, b, cc = _parts(s)
    y = s["tl"].scan(x, b, cc, s["dt"], s["a"], s["state"], s["batch"], d=s["d"], dt_bias=s["dt_bias"],
                     softplus=s["case"]["softplus"], workspace=s["workspace"])
    return {"y": y, "state": s["state"]}


def _plain_scan(s):
    c, begin, lens = s["case"], s["begin"].long(), _lengths(s["case"])
    x, b, cc = (m.float() for m in _parts(s))
    b, cc = (m.repeat_interleave(c["heads"] // c["groups"], 1) for m in (b, cc))
    dt = s["dt"].float()
    if s["dt_bias"] is not None:
        dt = dt + s["dt_bias"]
    if c["softplus"]:
        dt = torch.where(dt > 20, dt, torch.log1p(torch.exp(dt)))
    decay = torch.exp(dt * s["a"])
    u = dt[..., None] * x
    y = torch.empty_like(x)
    h = torch.zeros_like(s["state"][:c["seqs"]]) if c["fresh"] else s["state"][s["src"].long()]
    for t in range(max(lens)):
        m = sum(n > t for n in lens)  # the lengths do not increase: the first m sequences have a row t
        row = begin[:m] + t if m > 1 else slice(t, t + 1)
        h[:m].mul_(decay[row][..., None, None]).add_(b[row][..., None] * u[row][:, :, None])
        y[row] = (h[:m] * cc[row][..., None]).sum(2)
    if s["d"] is not None:
        y += s["d"][:, None] * x
    s["state"][s["dst"].long()] = h
    return {"y": y.to(torch.bfloat16), "state": s["state"]}


def _out(v, kind):
    """A row's values v: as bf16, or as 8-bit codes with one scale a row stand for them."""
    if kind == "bf16":
        return v.to(torch.bfloat16)
    scale = v.abs().amax(1, keepdim=True) / 127
    return (torch.round(v / scale).clamp(-127, 127) * scale).to(torch.bfloat16)


def _values(q, scale):
    return torch.mul(q, scale[:, None], out=torch.empty_like(q, dtype=torch.bfloat16))


def _own_gated(s):
    c, tl = s["case"], s["tl"]
    if c["out"] == "bf16":
        return {"y": tl.rmsnorm_gated(s["x"], s["z"], s["w"], EPS, group=c["group"], gate_first=c["first"])}
    return {"y": _values(*tl.rmsnorm_gated_s8(s["x"], s["z"], s["w"], EPS, group=c["group"], gate_first=c["first"]))}


def _plain_gated(s):
    c = s["case"]
    x, g = s["x"].float(), _silu(s["z"].float())
    u = (x * g if c["first"] else x).view(c["T"], -1, c["group"])
    v = (u / torch.sqrt((u * u).mean(2, keepdim=True) + EPS)).view(c["T"], c["K"]) * s["w"]
    return {"y": _out(v if c["first"] else v * g, c["out"])}


def _own_post(s):
    c, tl = s["case"], s["tl"]
    out = torch.empty_like(s["r"])  # not in place: every pass starts from the same stream
    if c["out"] == "bf16":
        y = tl.rmsnorm_post(s["x"], s["w_post"], s["r"], s["w"], EPS, scale=s["scale"], gate=s["gate"], residual_out=out)
    else:
        y = _values(*tl.rmsnorm_post_s8(s["x"], s["w_post"], s["r"], s["w"], EPS, scale=s["scale"], gate=s["gate"],
                                        residual_out=out))
    return {"y": y, "residual": out}


def _plain_post(s):
    x, r = s["x"].float(), s["r"]
    p = x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * s["w_post"] * s["scale"]
    if s["gate"] is not None:
        p = p * s["gate"]
    r = (r.float() + p).to(r.dtype)
    h = r.float()
    return {"y": _out(h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * s["w"], s["case"]["out"]), "residual": r}


# ------------------------------------------------------- in 64 bits, apart


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "gated": _exact_gated, "post": _exact_post}[case["op"]](s)


def _exact_conv(s):
    c, k = s["case"], s["case"]["width"]
    y = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    state = s["state"].double()
    at = 0
    for i, n in enumerate(_lengths(c)):
        rows = torch.cat((s["state"][int(s["src"][i])].double(), s["x"][at:at + n].double()), 0)
        win = rows.unfold(0, k, 1)[:n]  # [n, channels, width]
        out = (win * s["w"].double()).sum(2)
        if s["bias"] is not None:
            out = out + s["bias"].double()
        y[at:at + n] = out * torch.sigmoid(out) if c["act"] else out
        state[int(s["dst"][i])] = rows[rows.shape[0] - (k - 1):]
        at += n
    return {"y": y, "state": state}


def _exact_scan(s):
    """Blocks of 32 tokens: inside a block the sums over earlier tokens, the state at its start for the rest."""
    c, L = s["case"], 32
    hg = c["heads"] // c["groups"]
    inner, shared = c["heads"] * c["p"], c["groups"] * c["n"]
    dt = s["dt"].double()
    if s["dt_bias"] is not None:
        dt = dt + s["dt_bias"].double()
    if c["softplus"]:
        dt = torch.nn.functional.softplus(dt, threshold=50)
    rows = s["xbc"].shape[0]
    y = torch.empty((rows, c["heads"], c["p"]), dtype=torch.float64, device="cuda")
    state = s["state"].double()
    begin = s["begin"].tolist()
    for i in range(c["seqs"]):
        src = int(s["src"][i])
        S = s["state"][src].double() if src >= 0 else torch.zeros_like(state[0])
        for t in range(begin[i], begin[i + 1], L):
            m = s["xbc"][t:min(t + L, begin[i + 1])].double()
            n = m.shape[0]
            x = m[:, :inner].view(n, c["heads"], c["p"]).transpose(0, 1)
            B, C = (m[:, k:k + shared].view(n, c["groups"], c["n"]).transpose(0, 1).repeat_interleave(hg, 0)
                    for k in (inner, inner + shared))
            step = dt[t:t + n].T  # [heads, n]
            sums = torch.cumsum(step * s["a"].double()[:, None], 1)
            gap = (sums[:, :, None] - sums[:, None, :]).masked_fill(
                torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1), -math.inf)
            weights = (C @ B.mT) * torch.exp(gap) * step[:, None, :]
            out = weights @ x + torch.exp(sums)[..., None] * (C @ S)
            if s["d"] is not None:
                out = out + s["d"].double()[:, None, None] * x
            y[t:t + n] = out.transpose(0, 1)
            left = torch.exp(sums[:, -1:] - sums) * step
            S = torch.exp(sums[:, -1])[:, None, None] * S + (B * left[..., None]).mT @ x
        state[int(s["dst"][i])] = S
    return {"y": y, "state": state}


def _steps(v):
    step = v.abs().amax(1, keepdim=True) / 127
    return torch.round(v / step).clamp(-127, 127) * step


def _exact_gated(s):
    c = s["case"]
    z = s["z"].double()
    gate = z * torch.sigmoid(z)
    x = s["x"].double()
    if c["first"]:
        x = x * gate
    parts = []
    for k in range(0, c["K"], c["group"]):
        u = x[:, k:k + c["group"]]
        parts.append(u * torch.rsqrt(u.pow(2).mean(1, keepdim=True) + EPS) * s["w"][k:k + c["group"]].double())
    v = torch.cat(parts, 1)
    if not c["first"]:
        v = v * gate
    return {"y": v if c["out"] == "bf16" else _steps(v)}


def _exact_post(s):
    x = s["x"].double()
    p = x * torch.rsqrt(x.pow(2).mean(1, keepdim=True) + EPS) * s["w_post"].double()
    if s["gate"] is not None:
        p = p * s["gate"].double()
    r = s["r"].double() + s["scale"] * p
    h = r.to(s["r"].dtype).double()  # the norm is that of the stream as it is stored
    v = h * torch.rsqrt(h.pow(2).mean(1, keepdim=True) + EPS) * s["w"].double()
    return {"y": v if s["case"]["out"] == "bf16" else _steps(v), "residual": r}
