"""The recurrent block's operators on the GPU (tern_causal_conv, tern_scan,
tern_rmsnorm_gated, tern_rmsnorm_post) against the plain references of
recurrent_ref.py, within the bounds derived there."""
from __future__ import annotations

import numpy as np
import pytest

from tests import decoder_ref as dref
from tests import recurrent_ref as ref
from tests.test_gpu_decoder import operand_order

pytestmark = pytest.mark.gpu
F32 = np.float32
U = ref.U


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


@pytest.fixture(scope="module")
def tl(torch):
    import ternary_weight_linear_amd as tl
    tl.lib()
    return tl


def dev(torch, x, bf16=False):
    t = torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")
    return t.to(torch.bfloat16) if bf16 else t


def host(t):
    return t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def rounded(x, bf16):
    return dref.bf16(x) if bf16 else x.astype(F32)


def near(got, want, e, what=""):
    """bf16 outputs: the rounding of a value that is off by at most e."""
    bad = ~(np.abs(got - want) <= dref.half_ulp(np.abs(want) + e) + e)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def batch_of(torch, tl, begin, src, dst, max_q=None):
    most = max_q or max(1, max(b - a for a, b in zip(begin, begin[1:])))
    return tl.StateBatch(*(torch.tensor(v, dtype=torch.int32, device="cuda:0") for v in (begin, src, dst)), max_q=most)


# ------------------------------------------------------------ convolution

CONV_LENS = [[1], [2, 1, 3], [0, 5, 0, 17], [16, 33, 32], [509, 3, 64]]


@pytest.mark.parametrize("lens", CONV_LENS)
@pytest.mark.parametrize("width,bf16,ch,act,bias", [
    (4, False, 64, True, True), (4, True, 264, True, False), (3, False, 1032, False, True), (2, True, 8, True, True),
    (2, False, 40, True, False), (3, True, 2048, True, True)])
def test_conv(torch, tl, lens, width, bf16, ch, act, bias):
    rng = np.random.default_rng(ch * 31 + len(lens))
    begin = np.cumsum([0] + lens).tolist()
    rows, seqs, slots = begin[-1], len(lens), 2 * len(lens) + 1
    wide = rounded(rng.standard_normal((rows, ch + 24)), bf16)
    w, b = rounded(rng.standard_normal((ch, width)), bf16), rounded(rng.standard_normal(ch), bf16)
    pool = rounded(rng.standard_normal((slots, width - 1, ch)), bf16)
    order = rng.permutation(slots)
    src, dst = order[:seqs].copy(), order[seqs:2 * seqs]
    src[0] = -1 if seqs > 1 else slots  # neither is a slot: zeros
    x, state = dev(torch, wide, bf16)[:, 8:8 + ch], dev(torch, pool, bf16)
    out = torch.full((rows + 2, ch + 8), 7.0, dtype=torch.bfloat16, device="cuda:0")
    y = tl.causal_conv(x, dev(torch, w, bf16), state, batch_of(torch, tl, begin, src.tolist(), dst.tolist()),
                       bias=dev(torch, b, bf16) if bias else None, activation="silu" if act else None, out=out[:rows, :ch])
    assert tl.last_kernels() == ["causal_conv"]
    got, new = host(y), host(state)
    want_pool = pool.copy()
    for i, n in enumerate(lens):
        if n == 0:
            continue
        past = pool[src[i]] if 0 <= src[i] < slots else np.zeros_like(pool[0])
        want, kept, e = ref.conv(wide[begin[i]:begin[i + 1], 8:8 + ch].astype(np.float64), w.astype(np.float64),
                                 b.astype(np.float64) if bias else None, act, past)
        near(got[begin[i]:begin[i + 1]], want, e, i)
        want_pool[dst[i]] = kept
    assert np.array_equal(new, want_pool)  # inputs, as they are; other slots untouched
    o = host(out)
    assert (o[rows:] == 7).all() and (o[:, ch:] == 7).all()


def test_conv_in_pieces_and_in_place(torch, tl):
    """A prompt in pieces, its state in one slot, gives the bits of the whole."""
    rng = np.random.default_rng(3)
    n, ch, width = 70, 48, 4
    x, w = dev(torch, rng.standard_normal((n, ch)).astype(F32)), dev(torch, rng.standard_normal((ch, width)).astype(F32))
    whole = torch.zeros((2, width - 1, ch), device="cuda:0")
    y = tl.causal_conv(x, w, whole, batch_of(torch, tl, [0, n], [-1], [0]))
    state = torch.full_like(whole, 5.0)
    at, parts = 0, []
    for size in (1, 1, 2, 3, 16, 1, 31, 15):
        parts.append(tl.causal_conv(x[at:at + size], w, state, batch_of(torch, tl, [0, size], [-1 if at == 0 else 1], [1])))
        at += size
    assert at == n
    assert torch.equal(torch.cat(parts), y) and torch.equal(state[1], whole[0]) and (state[0] == 5).all()


def test_conv_keeps_bad_values_to_what_sees_them(torch, tl):
    rng = np.random.default_rng(4)
    lens, ch, width = [20, 20], 16, 4
    x = rng.standard_normal((40, ch)).astype(F32)
    x[5, 3], x[19, 2] = np.nan, np.inf
    state = torch.zeros((2, width - 1, ch), device="cuda:0")
    y = host(tl.causal_conv(dev(torch, x), dev(torch, np.ones((ch, width), F32)), state,
                            batch_of(torch, tl, [0, 20, 40], [-1, -1], [0, 1])))
    bad = np.zeros((40, ch), bool)
    bad[5:9, 3] = bad[19, 2] = True
    assert (np.isfinite(y) == ~bad).all()
    assert np.isfinite(host(state)[1]).all() and not np.isfinite(host(state)[0, 2, 2])


# ------------------------------------------------------------------- scan


class ScanCase:
    def __init__(self, torch, seed, lens, heads, groups, p, n, dt_bf16=False, bias=True, softplus=True, skip=True, slots=None,
                 strong=False):
        rng = np.random.default_rng(seed)
        self.lens, self.begin = lens, np.cumsum([0] + lens).tolist()
        rows = self.begin[-1]
        self.heads, self.groups, self.p, self.n, self.softplus = heads, groups, p, n, softplus
        width = heads * p + 2 * groups * n
        self.m = dref.bf16(rng.standard_normal((rows, width + 16)).astype(F32))
        self.x = self.m[:, :heads * p].reshape(rows, heads, p)
        self.b = self.m[:, heads * p:heads * p + groups * n].reshape(rows, groups, n)
        self.c = self.m[:, heads * p + groups * n:width].reshape(rows, groups, n)
        self.a = -rng.uniform(0.5, 16, heads).astype(F32)
        first = np.exp(rng.uniform(np.log(1e-3), np.log(1.0 if strong else 0.1), heads))
        dt = 0.5 * rng.standard_normal((rows, heads + 3))
        if softplus and bias:
            self.bias = (first + np.log(-np.expm1(-first))).astype(F32)
        else:
            self.bias, dt = None, np.log(np.expm1(first * np.exp(dt)[:, :1])) if softplus else first.mean() * np.exp(dt)
            dt = np.broadcast_to(dt, (rows, dt.shape[1]))[:, :heads]
            dt = np.concatenate((dt, np.zeros((rows, 3))), 1)
        self.dt = rounded(dt, dt_bf16)
        self.dt_bf16 = dt_bf16
        self.d = rng.standard_normal(heads).astype(F32) if skip else None
        seqs = len(lens)
        slots = slots or 2 * seqs + 1
        self.pool = rng.standard_normal((slots, heads, n, p)).astype(F32)
        order = rng.permutation(slots)
        self.src, self.dst = order[:seqs].tolist(), order[seqs:2 * seqs].tolist()

    def tensors(self, torch):
        m = dev(torch, self.m, True)
        rows, hp, gn = m.shape[0], self.heads * self.p, self.groups * self.n
        return dict(x=m[:, :hp].unflatten(1, (self.heads, self.p)), b=m[:, hp:hp + gn].unflatten(1, (self.groups, self.n)),
                    c=m[:, hp + gn:hp + 2 * gn].unflatten(1, (self.groups, self.n)),
                    dt=dev(torch, self.dt, self.dt_bf16)[:, :self.heads], a=dev(torch, self.a),
                    d=None if self.d is None else dev(torch, self.d),
                    dt_bias=None if self.bias is None else dev(torch, self.bias), softplus=self.softplus)

    def reference(self, i):
        r = slice(self.begin[i], self.begin[i + 1])
        s = self.pool[self.src[i]] if 0 <= self.src[i] < len(self.pool) else np.zeros_like(self.pool[0])
        return ref.Scan(self.x[r], self.b[r], self.c[r], self.dt[r, :self.heads], self.a.astype(np.float64), s,
                        None if self.d is None else self.d.astype(np.float64), self.bias, self.softplus)

    def check(self, y, state, left_out=()):
        want = self.pool.copy()
        for i, n in enumerate(self.lens):
            if n == 0 or i in left_out:
                continue
            r = self.reference(i)
            blocks = max(self.lens) > 8
            near(y[self.begin[i]:self.begin[i + 1]], r.y, r.y_bound(blocks), i)
            if 0 <= self.dst[i] < len(self.pool):
                got = state[self.dst[i]]
                e = r.s_bound(blocks) + U * np.abs(r.s)
                assert (np.abs(got - r.s) <= e).all(), (i, np.max(np.abs(got - r.s) / (np.abs(r.smag) + 1e-30)))
                want[self.dst[i]] = got
        assert np.array_equal(state, want)


def run_scan(torch, tl, c, **kw):
    state = dev(torch, c.pool)
    y = tl.scan(state=state, batch=batch_of(torch, tl, c.begin, c.src, c.dst, kw.pop("max_q", None)), **c.tensors(torch), **kw)
    return y, state


@pytest.mark.parametrize("p", [32, 64, 128])
@pytest.mark.parametrize("n", [64, 128, 256])
@pytest.mark.parametrize("lens,heads,groups", [([1], 3, 1), ([4, 1, 0, 3], 4, 2), ([8, 5], 2, 2)])
def test_scan_steps(torch, tl, p, n, lens, heads, groups):
    c = ScanCase(torch, p + n, lens, heads, groups, p, n)
    y, state = run_scan(torch, tl, c)
    assert tl.last_kernels() == ["scan_step"]
    c.check(host(y), host(state))


SCAN_LENS = [[9], [17], [31, 32, 33], [63, 64, 65], [1, 130, 0, 200], [509, 18]]


@pytest.mark.parametrize("lens", SCAN_LENS)
@pytest.mark.parametrize("p,n,heads,groups,kw", [
    (64, 128, 4, 2, {}), (32, 64, 10, 2, dict(dt_bf16=True)), (128, 256, 2, 1, dict(skip=False)),
    (64, 64, 3, 1, dict(softplus=False)), (32, 128, 5, 5, dict(bias=False)), (128, 128, 3, 1, dict(strong=True)),
    (64, 256, 5, 1, {}), (32, 256, 6, 2, {}), (128, 64, 2, 2, {})])
def test_scan_prompts(torch, tl, lens, p, n, heads, groups, kw):
    c = ScanCase(torch, p * n + sum(lens), lens, heads, groups, p, n, **kw)
    y, state = run_scan(torch, tl, c)
    assert tl.last_kernels() == ["scan_prepare", "scan_blocks"]
    c.check(host(y), host(state))


SEGMENTS = ["scan_blocks", "scan_join", "scan_prepare", "scan_states"]


@pytest.mark.parametrize("p,n,heads,groups,lens,place", [
    (64, 128, 2, 1, [2500, 0, 31, 700], "apart"), (32, 64, 5, 1, [1, 2049], "apart"), (128, 256, 1, 1, [1536], "in place"),
    (64, 64, 4, 2, [1601, 1600], "in place"), (32, 256, 2, 2, [1300, 1400], "from zeros"), (128, 64, 1, 1, [33, 4100], "in place")])
def test_scan_in_segments(torch, tl, p, n, heads, groups, lens, place):
    """Few heads and long prompts, which several workgroups share: each starts from its segment's state."""
    c = ScanCase(torch, p + n + heads, lens, heads, groups, p, n, slots=2 * len(lens) + 1)
    if place == "in place":
        c.dst = list(c.src)
    elif place == "from zeros":
        c.src[0], c.dst[1] = -1, -1
    y, state = run_scan(torch, tl, c)
    assert sorted(tl.last_kernels()) == SEGMENTS
    c.check(host(y), host(state))


def test_captured_segments(torch, tl):
    """A captured scan in segments, in place and replayed with other lengths, gives what eager calls give."""
    n = 1800
    c = ScanCase(torch, 18, [n, n], 2, 1, 64, 128)
    t, state = c.tensors(torch), dev(torch, c.pool)
    begin, slots = (torch.tensor(v, dtype=torch.int32, device="cuda:0") for v in (c.begin, c.src))
    batch = tl.StateBatch(begin, slots, slots, max_q=n)
    work = tl.scan_workspace(batch, 2 * n, 2, 64, 1, 128)
    out = torch.zeros((2 * n, 2, 64), dtype=torch.bfloat16, device="cuda:0")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        tl.scan(state=state, batch=batch, workspace=work, out=out, **t)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tl.scan(state=state, batch=batch, workspace=work, out=out, **t)
    assert sorted(tl.last_kernels()) == SEGMENTS
    for first, second in ((n, n), (1, n), (97, 0), (1000, 800)):
        begin.copy_(torch.tensor([0, first, first + second], dtype=torch.int32))
        state.copy_(dev(torch, c.pool)), out.zero_()
        work.fill_(255)  # any contents: NaN
        graph.replay()
        torch.cuda.synchronize()
        kept, mine = state.clone(), out.clone()
        state.copy_(dev(torch, c.pool)), out.zero_()
        tl.scan(state=state, batch=batch, out=out, **t)
        assert torch.equal(kept, state) and torch.equal(mine, out), (first, second)
        assert torch.isfinite(out).all() and (out[first + second:] == 0).all()
        assert torch.isfinite(state).all()


def test_scan_from_zeros_in_place_and_not_kept(torch, tl):
    for lens in ([3, 2, 4], [70, 100, 20]):
        c = ScanCase(torch, 9, lens, 4, 2, 64, 128)
        c.src[0], c.src[1], c.dst[2] = -1, len(c.pool), -7
        c.dst[1], free = c.src[2], c.dst[1]
        c.dst[1] = free
        y, state = run_scan(torch, tl, c)
        c.check(host(y), host(state))
        c = ScanCase(torch, 10, lens, 4, 2, 64, 128)
        c.dst = list(c.src)  # in place
        y, state = run_scan(torch, tl, c)
        c.check(host(y), host(state))


def test_scan_leaves_out_what_does_not_fit(torch, tl):
    """Offsets that fall, leave the rows or exceed max_q: rows, slot and neighbours stay as they were."""
    for n in (4, 40):
        c = ScanCase(torch, 11, [n, n, n], 2, 1, 64, 128)
        rows = 3 * n
        state = dev(torch, c.pool)
        out = torch.full((rows, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda:0")
        t = c.tensors(torch)
        for begin in ([0, n, rows + 1, rows + 1], [-1, n, n, n], [n, 0, n, n], [2 ** 31 - 1, -2 ** 31, n, n]):
            out.fill_(7.0), state.copy_(dev(torch, c.pool))
            tl.scan(state=state, batch=batch_of(torch, tl, begin, c.src, c.dst, max_q=n), out=out, **t)
            o, s = host(out), host(state)
            fits = [0 <= a < b <= rows and b - a <= n for a, b in zip(begin, begin[1:])]
            for i in range(3):
                assert (s[c.dst[i]] == c.pool[c.dst[i]]).all() == (not fits[i]), (begin, i)
            seen = np.zeros(rows, bool)
            for (a, b), f in zip(zip(begin, begin[1:]), fits):
                if f:
                    seen[a:b] = True
            assert ((o == 7).all((1, 2)) == ~seen).all(), begin
        tl.scan(state=state.copy_(dev(torch, c.pool)), batch=batch_of(torch, tl, c.begin, c.src, c.dst, max_q=n - 1),
                out=out.fill_(7.0), **t)
        assert (host(out) == 7).all() and np.array_equal(host(state), c.pool)


@pytest.mark.parametrize("n", [12, 90])
def test_scan_keeps_bad_values_to_what_sees_them(torch, tl, n):
    """A NaN or infinity in x, B, C, dt: earlier rows, other channels, heads, groups and sequences are as without it."""
    clean = ScanCase(torch, 12, [n, n], 4, 2, 64, 128)
    y0, s0 = (host(v) for v in run_scan(torch, tl, clean))
    t = n // 2 + 1
    for what, where, value in (("x", (t, 1, 5), np.nan), ("x", (t, 1, 5), np.inf), ("b", (t, 0, 7), np.nan),
                               ("c", (t, 1, 9), np.nan), ("dt", (t, 2), np.nan), ("dt", (t, 2), np.inf)):
        c = ScanCase(torch, 12, [n, n], 4, 2, 64, 128)
        getattr(c, what)[where] = value  # x, b and c are views of the matrix
        y, s = (host(v) for v in run_scan(torch, tl, c))
        see_y, see_s = np.zeros(y.shape, bool), np.zeros(s.shape, bool)
        if what == "x":
            see_y[t:n, 1, 5] = True
            see_s[c.dst[0], 1, :, 5] = True
        elif what == "b":
            see_y[t:n, :2] = True
            see_s[c.dst[0], :2, 7] = True
        elif what == "c":
            see_y[t, 2:] = True
        else:
            see_y[t:n, 2] = True
            see_s[c.dst[0], 2] = True
        assert np.array_equal(y[~see_y], y0[~see_y]), (what, value)
        assert np.array_equal(s[~see_s], s0[~see_s]), (what, value)
        assert not np.isfinite(y[see_y]).any() and not np.isfinite(s[see_s]).any(), (what, value)


def test_scan_forgets_at_a_large_step(torch, tl):
    """A step that takes the decay to zero (a document's end): what follows is
    as from zeros, with full precision of the steps after it."""
    n, t = 100, 37
    c = ScanCase(torch, 13, [n], 2, 1, 64, 128, softplus=False)
    c.dt[t] = 1e5
    c.x[t] = 0
    y, state = (host(v) for v in run_scan(torch, tl, c))
    r = ref.Scan(c.x[t + 1:], c.b[t + 1:], c.c[t + 1:], c.dt[t + 1:, :2], c.a.astype(np.float64), np.zeros_like(c.pool[0]),
                 c.d.astype(np.float64), None, False)
    # inside a block of 32 rows exponents are differences of sums up to 32 * 216 log(2): 4790 * 2^-24 and a few roundings each
    e = r.y_bound(True) + 2.0 ** -11 * r.ymag
    near(y[t + 1:], r.y, e)
    assert (np.abs(state[c.dst[0]] - r.s) <= r.s_bound(True) + 2.0 ** -11 * r.smag).all()


def test_scan_in_pieces(torch, tl):
    """A prompt in pieces, then tokens: each piece goes on from the state before it."""
    c = ScanCase(torch, 14, [230], 4, 2, 64, 128)
    t, state = c.tensors(torch), dev(torch, c.pool)
    want = c.reference(0)
    at, parts = 0, []
    for size in (128, 64, 17, 1, 4, 1, 15):
        step = {k: (v[at:at + size] if k in ("x", "b", "c", "dt") else v) for k, v in t.items()}
        parts.append(tl.scan(state=state, batch=batch_of(torch, tl, [0, size], [c.src[0] if at == 0 else c.dst[0]], [c.dst[0]]), **step))
        at += size
    assert at == 230
    near(host(torch.cat(parts)), want.y, want.y_bound(True))
    assert (np.abs(host(state)[c.dst[0]] - want.s) <= want.s_bound(True)).all()


@pytest.mark.parametrize("lens", [[3, 2], [40, 600]])
def test_offsets_past_32_bits(torch, tl, lens):
    """Slots behind 4 GiB of a pool and rows behind 4 GiB of x give the bits of small ones."""
    c = ScanCase(torch, 19, lens, 160, 8, 64, 128)
    t = c.tensors(torch)
    near_state = dev(torch, c.pool)
    y0 = tl.scan(state=near_state, batch=batch_of(torch, tl, c.begin, c.src, c.dst), **t)
    slots, rows = 900, c.begin[-1]
    far = torch.zeros((slots, 160, 128, 64), device="cuda:0")  # 4.7e9 bytes
    src, dst = [slots - 1, slots - 2], [slots - 3, slots - 4]
    for s, f in zip(c.src, src):
        far[f] = dev(torch, c.pool[s])
    step = 1 << 22  # the largest distance of rows: 640 of them pass 4 GiB
    x = torch.zeros(step * rows, dtype=torch.bfloat16, device="cuda:0").as_strided((rows, 160, 64), (step, 64, 1))
    t["x"] = x.copy_(t["x"])
    y = tl.scan(state=far, batch=batch_of(torch, tl, c.begin, src, dst), **t)
    assert torch.equal(y, y0)
    for d, f in zip(c.dst, dst):
        assert torch.equal(near_state[d], far[f])
    ch, slots = 16384, 24000
    z, w = torch.randn((rows, ch), device="cuda:0"), torch.randn((ch, 4), device="cuda:0")
    past = torch.randn((4, 3, ch), device="cuda:0")
    far = torch.zeros((slots, 3, ch), device="cuda:0")  # 4.7e9 bytes
    far[slots - 1], far[slots - 2] = past[0], past[1]
    o0 = tl.causal_conv(z, w, past, batch_of(torch, tl, c.begin, [0, 1], [2, 3]))
    o = tl.causal_conv(z, w, far, batch_of(torch, tl, c.begin, [slots - 1, slots - 2], [slots - 3, slots - 4]))
    assert torch.equal(o, o0) and torch.equal(far[slots - 3], past[2]) and torch.equal(far[slots - 4], past[3])


# ------------------------------------------------------------------ norms

GATED = [(1, 64, 64), (3, 48, 16), (7, 5120, 128), (5, 10240, 1280), (2, 960, 320), (4, 256, 256), (1, 32768, 32768),
         (3, 16448, 16448), (2, 20480, 64)]


@pytest.mark.parametrize("T,K,group", GATED)
@pytest.mark.parametrize("xt,zt,wt,first", [(0, 0, 0, True), (1, 0, 0, True), (1, 1, 1, False), (0, 1, 0, False)])
def test_gated_norm(torch, tl, T, K, group, xt, zt, wt, first):
    rng = np.random.default_rng(T * 7 + K)
    x, z = rounded(3 * rng.standard_normal((T, K)), xt), rounded(2 * rng.standard_normal((T, K + 16)), zt)
    w = rounded(1 + 0.2 * rng.standard_normal(K), wt)
    if T > 2:
        x[1, :group] = 0
        x[2] = 0
    if K > 200:
        z[0, :3] = (-200, 200, -87.5)
    want = ref.gated(x, z[:, 8:8 + K], w, 1e-6, group, first)
    xd, zd, wd = dev(torch, x, xt), dev(torch, z, zt)[:, 8:8 + K], dev(torch, w, wt)
    y = torch.full((T, K + 8), 7.0, dtype=torch.bfloat16, device="cuda:0")
    q, s = tl.rmsnorm_gated_s8(xd, zd, wd, 1e-6, group=group, gate_first=first, y=y[:, :K])
    assert tl.last_kernels() == ["rmsnorm_gated"]
    e = ref.GATED * np.abs(want) + 2.0 ** -100
    near(host(y)[:, :K], want, e)
    assert (host(y)[:, K:] == 7).all()
    step = np.abs(want).max(1) / 127
    assert (np.abs(host(s) - step) <= (ref.GATED + 2 * U) * step + 2.0 ** -100).all()
    q, s = host(q).astype(np.float64), host(s).astype(np.float64)
    # the quotient is within 127 * 2 * GATED of the exact one, the code half a step from it
    live = step > 0
    assert (np.abs(q[live] - want[live] / step[live, None]) <= 0.5 + 127 * (2 * ref.GATED + 4 * U)).all()
    assert (q[~live] == 0).all() and (s[~live] == 0).all()
    assert (np.abs(q[live]).max(1) == 127).all()
    y2 = tl.rmsnorm_gated(xd, zd, wd, 1e-6, group=group, gate_first=first)
    assert torch.equal(y2, y[:, :K])
    if group % 64 == 0:
        q2, s2 = tl.rmsnorm_gated_s8(xd, zd, wd, 1e-6, group=group, gate_first=first, layout="operand_order")
        assert np.array_equal(host(q2), operand_order(q.astype(np.int8))) and np.array_equal(host(s2), s.astype(F32))


def test_gated_norm_without_eps_and_bad_rows(torch, tl):
    rng = np.random.default_rng(8)
    x, z = rng.standard_normal((5, 256)).astype(F32), rng.standard_normal((5, 256)).astype(F32)
    x[0] = 0
    x[1, :64] = 0
    x[2, 70] = np.nan
    z[3, 70] = np.inf
    y = host(tl.rmsnorm_gated(dev(torch, x), dev(torch, z), torch.ones(256, device="cuda:0"), 0.0, group=64))
    want = ref.gated(x, z, np.ones(256), 0.0, 64, True)
    assert (y[0] == 0).all() and (y[1, :64] == 0).all()
    near(y[[1, 4]], want[[1, 4]], ref.GATED * np.abs(want[[1, 4]]))
    bad = np.zeros((5, 256), bool)
    bad[2, 64:128] = True
    assert np.isnan(y[2, 64:128]).all() and np.isfinite(y[~bad & (np.arange(5) != 3)[:, None]]).all()
    assert np.isfinite(y[3, :64]).all() and np.isfinite(y[3, 128:]).all() and not np.isfinite(y[3, 70])


POST = [(1, 16), (1, 5120), (5, 256), (3, 48), (17, 5120), (2, 16448), (2, 32768)]


@pytest.mark.parametrize("T,K", POST)
@pytest.mark.parametrize("xt,rt,wt,gate", [(0, 0, 0, None), (1, 1, 0, "channels"), (0, 1, 1, "tokens"), (1, 0, 0, "tokens")])
def test_post_norm(torch, tl, T, K, xt, rt, wt, gate):
    rng = np.random.default_rng(T * 11 + K)
    x, r = rounded(3 * rng.standard_normal((T, K + 16)), xt), rounded(2 * rng.standard_normal((T, K)), rt)
    pw, w = rounded(1 + 0.2 * rng.standard_normal(K), wt), rounded(1 + 0.2 * rng.standard_normal(K), wt)
    g = None if gate is None else rounded(rng.standard_normal(K if gate == "channels" else (T, K)), xt)
    if T > 2:
        x[1] = 0
    want, e = ref.post(x[:, 8:8 + K], pw, r, 0.37, g, 1e-6)
    xd, rd, pd, wd = dev(torch, x, xt)[:, 8:8 + K], dev(torch, r, rt), dev(torch, pw, wt), dev(torch, w, wt)
    gd = None if g is None else dev(torch, g, xt)
    ro = torch.full((T, K + 8), 7.0, dtype=rd.dtype, device="cuda:0")
    y = torch.empty((T, K), dtype=torch.bfloat16, device="cuda:0")
    q, s = tl.rmsnorm_post_s8(xd, pd, rd, wd, 1e-6, scale=0.37, gate=gd, residual_out=ro[:, :K], y=y)
    assert tl.last_kernels() == ["rmsnorm_post"]
    h = host(ro)[:, :K]
    if rt:
        near(h, want, e)
    else:
        assert (np.abs(h - want) <= e).all()
    assert (host(ro)[:, K:] == 7).all() and np.array_equal(host(rd), r)
    # the second norm is that of the stream as it was stored: codes to the bit
    y64, _, q_ref, s_ref = dref.rmsnorm(h, w, 1e-6)
    assert np.array_equal(host(q), q_ref)
    assert np.all(np.abs(host(s).astype(np.float64) - s_ref) <= 32 * U * s_ref)
    near(host(y), y64, 32 * U * np.abs(y64))
    r2 = rd.clone()
    y2 = tl.rmsnorm_post(xd, pd, r2, wd, 1e-6, scale=0.37, gate=gd)  # in place
    assert torch.equal(y2, y) and torch.equal(r2, ro[:, :K])
    r3 = rd.clone()
    assert tl.rmsnorm_post(xd, pd, r3, eps=1e-6, scale=0.37, gate=gd) is None and torch.equal(r3, r2)
    if K % 64 == 0:
        q2, s2 = tl.rmsnorm_post_s8(xd, pd, rd.clone(), wd, 1e-6, scale=0.37, gate=gd, layout="operand_order")
        assert np.array_equal(host(q2), operand_order(q_ref)) and torch.equal(s2, s)


# -------------------------------------------------- streams, graphs, refusals


def test_on_another_stream(torch, tl):
    c = ScanCase(torch, 15, [40, 3], 4, 2, 64, 128)
    y0, s0 = run_scan(torch, tl, c)
    t, state, batch = c.tensors(torch), dev(torch, c.pool), batch_of(torch, tl, c.begin, c.src, c.dst)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = tl.scan(state=state, batch=batch, stream=side, **t)
    side.synchronize()
    assert torch.equal(y, y0) and torch.equal(state, s0)


@pytest.mark.parametrize("n", [2, 80])
def test_captured_calls_follow_their_arrays(torch, tl, n):
    """A captured convolution, scan and gated norm, replayed with new inputs,
    offsets and slots, give what eager calls give."""
    c = ScanCase(torch, 16, [n, n], 4, 2, 64, 128)
    t, state = c.tensors(torch), dev(torch, c.pool)
    begin, src, dst = (torch.tensor(v, dtype=torch.int32, device="cuda:0") for v in (c.begin, c.src, c.dst))
    batch = tl.StateBatch(begin, src, dst, max_q=n)
    work = tl.scan_workspace(batch, 2 * n, 4, 64, 2, 128)
    z = torch.randn((2 * n, 256), device="cuda:0")
    weight, past = torch.randn((256, 4), device="cuda:0"), torch.randn((5, 3, 256), device="cuda:0")
    ones = torch.ones(256, device="cuda:0")

    def step():
        y = tl.scan(state=state, batch=batch, workspace=work, **t)
        o = tl.causal_conv(z, weight, past, batch)
        return y, o, tl.rmsnorm_gated(y.flatten(1), z, ones, group=64)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for k in range(4):
        begin.copy_(torch.tensor([0, n - k % 2, 2 * n], dtype=torch.int32))
        begin[2] = 2 * n - k % 2 if k < 3 else 2 * n
        src.copy_(torch.tensor([c.src[k % 2], c.src[1 - k % 2]], dtype=torch.int32))
        z.normal_()
        state.copy_(dev(torch, c.pool))
        past.fill_(0.5 * k)
        graph.replay()
        torch.cuda.synchronize()
        mine, kept, inputs = [v.clone() for v in got], state.clone(), past.clone()
        state.copy_(dev(torch, c.pool))
        past.fill_(0.5 * k)
        ends = begin.tolist()
        rows = ends[2] if ends[2] - ends[1] <= n else ends[1]  # the last replay's second sequence exceeds max_q
        want = step()
        for a, b in zip(mine, want):
            assert torch.equal(a[:rows], b[:rows]), k
        assert torch.equal(kept, state) and torch.equal(inputs, past)


def test_binding_refuses(torch, tl):
    c = ScanCase(torch, 17, [4], 4, 2, 64, 128)
    t, state, batch = c.tensors(torch), dev(torch, c.pool), batch_of(torch, tl, c.begin, c.src, c.dst)
    bad = [dict(b=t["b"][:, :1].contiguous()), dict(dt=t["dt"][:, :3]), dict(a=t["a"][:3]), dict(x=t["x"].float()),
           dict(c=t["c"][:3]), dict(state=state[:, :, :64]), dict(d=t["d"].double()), dict(dt=t["dt"].t().contiguous().t()),
           dict(a=t["a"].cpu()), dict(out=torch.empty((4, 4, 32), dtype=torch.bfloat16, device="cuda:0"))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, tl.TernError)):
            tl.scan(**{**t, "state": state, "batch": batch, **kw})
    x, w = torch.randn((4, 64), device="cuda:0"), torch.randn((64, 4), device="cuda:0")
    past = torch.zeros((3, 3, 64), device="cuda:0")
    for args, kw in (((x, w, past.bfloat16(), batch), {}), ((x, w[:, :3], past, batch), {}), ((x, w, past[:, :2], batch), {}),
                     ((x, w, past, batch), dict(activation="relu")), ((x, w, past, batch), dict(bias=w[:, 0])),
                     ((x[:, :60], w[:60], past[:, :, :60], batch), {}), ((x, w, past, batch), dict(out=x))):
        with pytest.raises((ValueError, TypeError, tl.TernError)):
            tl.causal_conv(*args, **kw)
    xb = x.bfloat16()
    with pytest.raises(tl.TernError):
        tl.causal_conv(xb, w, past.bfloat16(), batch, out=xb)
    with pytest.raises(ValueError):
        tl.StateBatch(batch.begin, batch.src, batch.dst, max_q=2 ** 31)
    with pytest.raises(tl.TernError):
        tl.rmsnorm_gated(x, x, torch.ones(64, device="cuda:0"), group=48)
    with pytest.raises(ValueError):
        tl.rmsnorm_post(x, torch.ones(64, device="cuda:0"), x, y=xb)
    with pytest.raises(ValueError):
        tl.rmsnorm_post(x, torch.ones(64, device="cuda:0"), x[:2])
