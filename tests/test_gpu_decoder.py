"""The decoder operators on the GPU (tern_rmsnorm, tern_kv_append, tern_kv_read,
tern_kv_attn) against the plain references of decoder_ref.py: codes, scales of
pages and residuals bit for bit, the rest within bounds derived there."""
from __future__ import annotations

import numpy as np
import pytest

from tests import decoder_ref as ref

pytestmark = pytest.mark.gpu
F32 = np.float32


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


def to_dev(torch, x, bf16=False):
    t = torch.from_numpy(np.ascontiguousarray(x)).to("cuda:0")
    return t.to(torch.bfloat16) if bf16 else t


def host(t):
    return t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def outliers(rng, shape):
    x = rng.standard_normal(shape).astype(F32)
    x[..., rng.random(shape[-1]) < 0.01] *= 20
    return x


# ------------------------------------------------------------------- norm


def operand_order(q):
    """Row-major codes [T, K] in the s8 contraction's byte order."""
    T, K = q.shape
    out = np.empty_like(q)
    at = np.arange(K)
    blk, rest = at // 64, at % 64
    g, i, e = rest // 16, rest % 16 // 4, rest % 4
    m = np.array([[32 + 2 * j, 2 * j, 33 + 2 * j, 2 * j + 1] for j in range(4)])
    out[:] = q[:, 64 * blk + 8 * g + m[i, e]]
    return out


NORM_SIZES = [(1, 16), (1, 5120), (3, 256), (7, 48), (17, 1024), (33, 5120), (2, 16384), (2, 16448), (5, 32768)]


@pytest.mark.parametrize("T,K", NORM_SIZES)
@pytest.mark.parametrize("xt,rt,wt", [(0, 0, 0), (0, 1, 1), (1, 1, 0), (1, None, 1), (0, None, 0), (1, 0, 1)])
def test_rmsnorm(torch, tl, T, K, xt, rt, wt):
    rng = np.random.default_rng(T * 100003 + K)
    x, w = outliers(rng, (T, K)), (1 + 0.2 * rng.standard_normal(K)).astype(F32)
    r = outliers(rng, (T, K)) * 3
    x, w, r = (ref.bf16(a) if t == 1 else a for a, t in ((x, xt), (w, wt), (r, rt)))
    y64, h, q_ref, s_ref = ref.rmsnorm(x, w, 1e-6, None if rt is None else r, rt == 1)
    xd, wd = to_dev(torch, x, xt == 1), to_dev(torch, w, wt == 1)
    rd = None if rt is None else to_dev(torch, r, rt == 1)
    ro = None if rt is None else torch.empty_like(rd)
    y = torch.empty((T, K), dtype=torch.bfloat16, device="cuda:0")
    q, s = tl.rmsnorm_s8(xd, wd, 1e-6, residual=rd, residual_out=ro, y=y)
    assert tl.last_kernels() == ["rmsnorm"]
    assert np.array_equal(host(q), q_ref)
    # rho: at most 32 + 4 + 16 roundings of a sum of squares (half of them
    # after the root), the division, the root and two products: under 32 ulp
    assert np.all(np.abs(host(s).astype(np.float64) - s_ref) <= 32 * 2.0 ** -24 * s_ref)
    e = 32 * 2.0 ** -24 * np.abs(y64)
    assert np.all(np.abs(host(y) - y64) <= ref.half_ulp(np.abs(y64) + e) + e)
    if rt is not None:
        assert np.array_equal(host(ro), h)
        assert np.array_equal(host(rd), r)  # not in place
        y2 = tl.rmsnorm(xd, wd, 1e-6, residual=rd)  # in place
        assert np.array_equal(host(rd), h) and torch.equal(y2, y)
    if K % 64 == 0:
        q2, s2 = tl.rmsnorm_s8(xd, wd, 1e-6, residual=None if rt is None else to_dev(torch, r, rt == 1),
                               layout="operand_order")
        assert np.array_equal(host(q2), operand_order(q_ref)) and torch.equal(s2, s)


def test_rmsnorm_rows_apart_and_special_rows(torch, tl):
    """Rows inside wider matrices; rows of zeros, of one value, of subnormals;
    a NaN or infinity stays in its row."""
    rng = np.random.default_rng(5)
    T, K = 9, 512
    wide = outliers(rng, (T, K + 64))
    wide[1] = 0
    wide[2] = 3.5
    wide[3, 32:32 + K] = 1e-41
    wide[4, 100] = np.nan
    wide[5, 100] = np.inf
    wide[6] *= 1e15
    x = to_dev(torch, wide)[:, 32:32 + K]
    res = torch.zeros((T, 2 * K), dtype=torch.float32, device="cuda:0")
    out = torch.full((T, 3 * K), 7.0, dtype=torch.float32, device="cuda:0")
    y = torch.full((T, K + 8), 7.0, dtype=torch.bfloat16, device="cuda:0")
    w = torch.ones(K, device="cuda:0")
    q, s = tl.rmsnorm_s8(x, w, 1e-6, residual=res[:, K:], residual_out=out[:, K:2 * K], y=y[:, :K])
    xs = wide[:, 32:32 + K]
    fine = [0, 1, 2, 3, 6, 7, 8]
    y64, h, q_ref, s_ref = ref.rmsnorm(xs[fine], np.ones(K, F32), 1e-6)
    assert np.array_equal(host(q)[fine], q_ref)
    assert np.all(np.abs(host(s)[fine] - s_ref) <= 32 * 2.0 ** -24 * s_ref + 2.0 ** -149)
    e = 32 * 2.0 ** -24 * np.abs(y64) + 2.0 ** -149
    assert np.all(np.abs(host(y)[fine, :K] - y64) <= ref.half_ulp(np.abs(y64) + e) + e)
    assert np.isnan(host(s)[4]) and not np.isfinite(host(s)[5])
    o = host(out)
    assert np.array_equal(o[fine, K:2 * K], xs[fine])
    assert np.all(o[:, :K] == 7) and np.all(o[:, 2 * K:] == 7) and np.all(host(y)[:, K:] == 7)


def test_rmsnorm_feeds_the_s8_contraction(torch, tl):
    """(q, scale) of the norm through linear_s8_q: the layer on the norm's
    dequantised output, both byte orders the same."""
    rng = np.random.default_rng(11)
    T, K, N, G = 19, 512, 48, 128
    w = rng.integers(-1, 2, (N, K)).astype(np.int8)
    sc = rng.uniform(0.01, 0.05, (N, K // G)).astype(np.float16)
    W = tl.TernaryWeights.from_host(w, sc, device="cuda:0")
    x, g = outliers(rng, (T, K)), (1 + 0.1 * rng.standard_normal(K)).astype(F32)
    _, _, q_ref, s_ref = ref.rmsnorm(x, g, 1e-6)
    want = (q_ref.astype(np.float64) * s_ref[:, None]) @ (w * np.repeat(sc.astype(np.float64), G, 1)).T
    for layout in ("row_major", "operand_order"):
        q, s = tl.rmsnorm_s8(to_dev(torch, x), to_dev(torch, g), 1e-6, layout=layout)
        y = host(tl.linear_s8_q(q, s, W, layout=layout))
        # scale: 32 ulp; the contraction's fp32 epilogue: K/G + 2 roundings of the absolute sum
        mag = (np.abs(q_ref).astype(np.float64) * s_ref[:, None]) @ np.abs(w * np.repeat(sc.astype(np.float64), G, 1)).T
        assert np.all(np.abs(y - want) <= (32 + K // G + 4) * 2.0 ** -24 * mag)


# ------------------------------------------------------------------ cache


def make_rope(rng, positions, pairs, axes):
    f = 1e4 ** (-np.arange(pairs) / pairs)
    a = np.arange(positions)[:, None] * f
    return np.stack((np.cos(a), np.sin(a)), -1).astype(F32), rng.integers(0, axes, pairs).astype(np.uint8)


def new_table(rng, pages, needs):
    """Pages of random order for sequences that need so many; width a little larger."""
    order = rng.permutation(pages).astype(np.int32)
    t = np.full((len(needs), max(max(needs), 1) + 1), -1, np.int32)
    at = 0
    for i, n in enumerate(needs):
        t[i, :n] = order[at:at + n]
        at += n
    assert at <= pages
    return t


def batch_of(torch, tl, ns, lens, table, max_q=None, max_kv=None):
    q_begin = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
    return tl.KVBatch(to_dev(torch, q_begin), to_dev(torch, np.asarray(lens, np.int32)), to_dev(torch, table),
                      max(max(ns), 1) if max_q is None else max_q, max(max(lens), 1) if max_kv is None else max_kv)


def device_codes(cache):
    k = host(cache.k)
    v = host(cache.v)[..., ref.PLACES].transpose(0, 1, 3, 2)
    return k, v


def check_cache(cache, model, tables, lens):
    """Codes of every token that is stored and scales of its pages, bit for bit."""
    k, v = device_codes(cache)
    ks, vs = host(cache.k_scale), host(cache.v_scale)
    for table, n in zip(tables, lens):
        for p in range((n + 63) // 64):
            m = min(64, n - 64 * p)
            for got, sc, which in ((k, ks, 0), (v, vs, 1)):
                assert np.array_equal(sc[table[p]], model.s[which][table[p]])
                assert np.array_equal(got[table[p], :, :m], model.c[which][table[p], :, :m]), (p, which)


@pytest.mark.parametrize("d,heads,group,pairs,axes,bf16", [
    (64, 1, 1, 32, 1, False), (128, 2, 5, 64, 3, False), (128, 8, 1, 32, 3, True), (256, 2, 3, 128, 3, True),
    (256, 1, 4, 4, 2, False), (64, 3, 2, 0, 1, True)])
def test_append_grows_pages(torch, tl, d, heads, group, pairs, axes, bf16):
    """A run of calls on ragged sequences: prompts that end inside pages, single
    tokens, sequences without tokens in a call, values that grow and shrink, a
    token of zeros. Codes and scales after every call, q and the read-out too."""
    rng = np.random.default_rng(d + heads * 7 + pairs)
    calls = [[5, 64, 0, 130], [1, 1, 1, 1], [0, 63, 70, 1], [60, 1, 1, 64], [1, 0, 0, 1], [2, 3, 4, 5]]
    size = [1.0, 0.1, 3.0, 1.0, 40.0, 0.0]
    total = np.sum(calls, 0)
    pages = int(((total + 63) // 64).sum()) + 2
    table = new_table(rng, pages, [int(x) for x in (total + 63) // 64])
    cache, model = tl.KVCache.empty(pages, heads, d, "cuda:0"), ref.Cache(pages, heads, d)
    cache.k.fill_(-128)  # slots that hold nothing may hold anything
    cache.v.fill_(-128)
    rt, axis = make_rope(rng, 300, max(pairs, 4), axes)
    turn = tl.Rope(to_dev(torch, rt), to_dev(torch, axis)) if pairs else None
    hq = heads * group
    lens = np.zeros(4, int)
    for ns, mul in zip(calls, size):
        tokens = sum(ns)
        x = outliers(rng, (tokens, hq + 2 * heads, d)) * F32(mul)
        if bf16:
            x = ref.bf16(x)
        positions = rng.integers(-2, 305, (axes, tokens)).astype(np.int32)  # clamped to the table
        t = (lambda z: ref.rope(z, rt, axis, positions)) if pairs else (lambda z: z)
        lens = lens + ns
        row = 0
        for s, n in enumerate(ns):
            if n:
                sl = slice(row, row + n)
                model.append(table[s], lens[s] - n, t(x[:, hq:hq + heads])[sl], x[sl, hq + heads:])
            row += n
        xd = to_dev(torch, x, bf16)
        b = batch_of(torch, tl, ns, lens, table, max_q=max(ns) + 3, max_kv=int(max(lens)) + 9)
        q = tl.kv_append(cache, b, xd[:, hq:hq + heads], xd[:, hq + heads:], q=xd[:, :hq], rope=turn,
                         positions=to_dev(torch, positions) if pairs else None)
        assert tl.last_kernels() == ["kv_append"]
        check_cache(cache, model, table, lens)
        assert np.array_equal(host(q), ref.bf16(t(x[:, :hq])))
        last = [min(int(n), 70) for n in lens]
        rb = batch_of(torch, tl, last, lens, table)
        k, v = tl.kv_read(cache, rb, sum(last))
        for which, got in ((0, k), (1, v)):
            want = np.concatenate([model.values(which, table[s], n - m, n) for s, (n, m) in enumerate(zip(lens, last))])
            assert np.array_equal(host(got), ref.bf16(want.astype(F32)))  # fl(code * scale), then bf16
    # nothing outside the sequences' pages was written
    used = set(table[table >= 0].tolist())
    for p in set(range(pages)) - used:
        assert (cache.k[p] == -128).all() and (cache.v[p] == -128).all()


def test_append_leaves_out_what_contradicts_its_bounds(torch, tl):
    """Pages outside the cache, rows past the tokens, more tokens than max_q or
    than the sequence holds: nothing is written for those sequences."""
    rng = np.random.default_rng(3)
    d, heads, pages = 64, 2, 6
    cache, model = tl.KVCache.empty(pages, heads, d, "cuda:0"), ref.Cache(pages, heads, d)
    k, v = outliers(rng, (12, heads, d)), outliers(rng, (12, heads, d))
    table = np.array([[0, 1], [99, 2], [-5, 3], [4, 5]], np.int32)
    qb = np.array([0, 3, 6, 9, 12], np.int32)
    b = tl.KVBatch(to_dev(torch, qb), to_dev(torch, np.array([3, 3, 3, 2], np.int32)), to_dev(torch, table), 3, 128)
    tl.kv_append(cache, b, to_dev(torch, k), to_dev(torch, v))
    model.append(table[0], 0, k[:3], v[:3])
    check_cache(cache, model, table[:1], [3])
    for p in range(1, 6):
        assert not cache.k[p].any() and not cache.v[p].any() and not cache.k_scale[p].any()
    before = cache.k.clone(), cache.v.clone(), cache.k_scale.clone()
    for qb, kv in (([0, 4, 4, 4, 4], [64] * 4), ([0, 3, 14, 14, 14], [0, 200, 0, 0]), ([-3, 0, 0, 0, 0], [64] * 4),
                   ([3, 0, 0, 0, 0], [64] * 4)):
        b = tl.KVBatch(to_dev(torch, np.array(qb, np.int32)), to_dev(torch, np.array(kv, np.int32)),
                       to_dev(torch, table), 3, 128)
        tl.kv_append(cache, b, to_dev(torch, k), to_dev(torch, v))
        for x, y in zip(before, (cache.k, cache.v, cache.k_scale)):
            assert torch.equal(x, y)


def test_append_nan_stays_in_its_page_and_head(torch, tl):
    rng = np.random.default_rng(4)
    d, heads = 64, 2
    cache = tl.KVCache.empty(3, heads, d, "cuda:0")
    k, v = outliers(rng, (130, heads, d)), outliers(rng, (130, heads, d))
    k[70, 1, 3], v[5, 0, 9] = np.nan, np.inf
    table = np.array([[2, 0, 1]], np.int32)
    tl.kv_append(cache, batch_of(torch, tl, [130], [130], table), to_dev(torch, k), to_dev(torch, v))
    model = ref.Cache(3, heads, d)
    with np.errstate(all="ignore"):
        model.append(table[0], 0, np.nan_to_num(k, nan=0), np.nan_to_num(v, posinf=0))
    ks, vs = host(cache.k_scale), host(cache.v_scale)
    assert np.isnan(ks[0, 1]) and np.isinf(vs[2, 0])
    ks[0, 1], vs[2, 0] = model.s[0][0, 1], model.s[1][2, 0]
    assert np.array_equal(ks, model.s[0]) and np.array_equal(vs, model.s[1])


# -------------------------------------------------------------- attention


class Filled:
    """A cache filled through the model (random codes and scales), and its
    sequences; unused slots and pages hold the worst bytes, and the scales of
    unused pages are NaN."""

    def __init__(self, torch, tl, rng, lens, heads, d, spread=1.0, extra=3):
        needs = [(n + 63) // 64 for n in lens]
        pages = sum(needs) + extra
        self.table = new_table(rng, pages, needs)
        self.model = ref.Cache(pages, heads, d)
        self.lens = lens
        for s, n in enumerate(lens):
            for p in range(needs[s]):
                x = rng.standard_normal((2, min(64, n - 64 * p), heads, d)).astype(F32)
                x[1] *= F32(spread) ** rng.integers(-3, 4, (1, heads, 1)).astype(F32)
                self.model.append(self.table[s][p:], 0, x[0], x[1])
        k, v = np.full((pages, heads, 64, d), -128, np.int8), np.full((pages, heads, d, 64), -128, np.int8)
        ks, vs = np.full((pages, heads), np.nan, F32), np.full((pages, heads), np.nan, F32)
        for s, n in enumerate(lens):
            for p in range(needs[s]):
                m, pg = min(64, n - 64 * p), self.table[s][p]
                k[pg, :, :m] = self.model.c[0][pg, :, :m]
                v[pg][:, :, ref.PLACES[:m]] = self.model.c[1][pg, :, :m].transpose(0, 2, 1)
                ks[pg], vs[pg] = self.model.s[0][pg], self.model.s[1][pg]
        self.cache = tl.KVCache(*(to_dev(torch, a) for a in (k, v, ks, vs)))

    def kv(self, s):
        n = self.lens[s]
        return [self.model.values(w, self.table[s], 0, n) for w in (0, 1)]


def check_attention(f, q, out, ns, scale, window=0, sinks=0, d=None):
    row = 0
    out = host(out).astype(np.float64)
    for s, n in enumerate(ns):
        k, v = f.kv(s)
        want, mag, top = ref.attention(q[row:row + n].astype(np.float64), k, v, f.lens[s] - n, scale, window, sinks)
        bound = ref.attention_bound(want, mag, top, q.shape[2])
        bad = np.abs(out[row:row + n] - want) > bound
        assert not bad.any(), (s, np.argwhere(bad)[:4], np.abs(out[row:row + n] - want)[bad][:4], bound[bad][:4])
        row += n


ATTN = [
    # d, kv heads, group, tokens of the call, lengths, window, sinks
    (128, 2, 5, [1], [1], 0, 0),
    (128, 1, 1, [1, 1, 1], [63, 64, 65], 0, 0),
    (64, 2, 8, [1, 1, 1, 1], [1, 200, 1000, 2], 0, 0),
    (256, 1, 6, [1, 1], [129, 700], 0, 0),
    (128, 2, 5, [4, 1, 0, 3], [4, 500, 77, 3], 0, 0),
    (64, 1, 3, [7, 70], [9, 300], 0, 0),
    (128, 1, 16, [3], [400], 0, 0),
    (64, 1, 17, [5, 2], [64, 128], 0, 0),
    (128, 1, 40, [2], [90], 0, 0),
    (256, 2, 2, [33], [100], 0, 0),
    (128, 2, 1, [130], [130], 0, 0),
    (128, 1, 5, [65, 1], [321, 64], 0, 0),
    (64, 2, 4, [1, 1, 1], [1000, 300, 10], 100, 0),
    (64, 2, 4, [1, 1, 1], [1000, 300, 10], 100, 4),
    (128, 1, 5, [50, 3], [700, 64], 64, 65),
    (128, 1, 2, [90], [600], 1, 0),
    (256, 1, 3, [20, 5], [900, 6], 33, 128),
    (128, 1, 4, [100], [100], 1000, 2),
]


@pytest.mark.parametrize("d,heads,group,ns,lens,window,sinks", ATTN)
def test_attention(torch, tl, d, heads, group, ns, lens, window, sinks):
    rng = np.random.default_rng(d * 1000 + sum(lens) + group)
    f = Filled(torch, tl, rng, lens, heads, d)
    q = ref.bf16(rng.standard_normal((sum(ns), heads * group, d)).astype(F32) * F32(1.5))
    b = batch_of(torch, tl, ns, lens, f.table)
    out = tl.kv_attn(to_dev(torch, q, True), f.cache, b, d ** -0.5, window=window, sinks=sinks)
    check_attention(f, q, out, ns, d ** -0.5, window, sinks)


@pytest.mark.parametrize("n,window,sinks", [(1, 0, 0), (3, 0, 0), (1, 5000, 7), (40, 0, 0)])
def test_attention_long_and_split(torch, tl, n, window, sinks):
    """Key axes long enough to be cut into runs; bounds larger than the lengths;
    sequences whose runs are partly or wholly empty; large scores, so that a
    few keys hold most of the weight; value scales of very different size."""
    rng = np.random.default_rng(n + window)
    lens, ns = [9000, 64 * 20 + 1, n], [n, n, n]
    f = Filled(torch, tl, rng, lens, 1, 128, spread=30.0)
    q = ref.bf16(rng.standard_normal((3 * n, 5, 128)).astype(F32) * F32(4))
    b = batch_of(torch, tl, ns, lens, f.table, max_q=n + 2, max_kv=f.table.shape[1] * 64)
    ws = tl.kv_attn_workspace(f.cache, b, 3 * n, 5, window, sinks)
    assert ws is not None
    ws.fill_(255)  # NaN
    out = tl.kv_attn(to_dev(torch, q, True), f.cache, b, 128 ** -0.5, window=window, sinks=sinks, workspace=ws)
    assert "kv_attn_join" in tl.last_kernels()
    check_attention(f, q, out, ns, 128 ** -0.5, window, sinks)
    again = tl.kv_attn(to_dev(torch, q, True), f.cache, b, 128 ** -0.5, window=window, sinks=sinks, workspace=ws)
    assert torch.equal(out, again)


def test_attention_rows_that_see_nothing(torch, tl):
    """Lengths of zero, queries before the first key, pages outside the cache:
    zeros, and NaN scales behind them do not come through."""
    rng = np.random.default_rng(8)
    f = Filled(torch, tl, rng, [100, 3, 130], 2, 64)
    q = ref.bf16(rng.standard_normal((11, 4, 64)).astype(F32))
    ns = [1, 5, 1, 4]
    table = np.concatenate((f.table, np.full((1, f.table.shape[1]), 10 ** 6, np.int32)))
    table[2, 1] = -7  # the middle page of the third sequence is absent
    qb = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
    b = tl.KVBatch(to_dev(torch, qb), to_dev(torch, np.array([0, 3, 130, 128], np.int32)), to_dev(torch, table), 5, 192)
    out = host(tl.kv_attn(to_dev(torch, q, True), f.cache, b, 0.125)).astype(np.float64)
    assert not out[0].any()          # no keys
    assert not out[1:3].any()        # positions -2 and -1
    assert not out[7:].any()         # no page exists
    k, v = f.kv(1)
    want, mag, top = ref.attention(q[3:6].astype(np.float64), k, v, 0, 0.125)
    assert np.all(np.abs(out[3:6] - want) <= ref.attention_bound(want, mag, top, 64))
    k, v = f.kv(2)
    present = np.ones(130, bool)
    present[64:128] = False
    want, mag, top = ref.attention(q[6:7].astype(np.float64), k, v, 129, 0.125, present=present)
    assert np.all(np.abs(out[6:7] - want) <= ref.attention_bound(want, mag, top, 64))


def test_attention_special_values(torch, tl):
    """Queries of zeros, huge, tiny and subnormal; a NaN in a query or a page's
    scale reaches exactly the rows that see it; a page of zero values; tiny
    value scales keep their share of the sum."""
    rng = np.random.default_rng(9)
    f = Filled(torch, tl, rng, [300, 300], 1, 128)
    for which, page, s in ((1, f.table[0][1], 0.0), (1, f.table[0][2], 2.0 ** -90)):
        f.model.s[which][page] = s
        f.cache.v_scale[int(page)] = s
    f.model.c[1][f.table[0][1]] = 0
    f.cache.v[int(f.table[0][1])] = 0
    q = ref.bf16(rng.standard_normal((10, 2, 128)).astype(F32))
    q[0, 0] = 0
    q[1, 0] *= F32(2.0 ** 100)
    q[2, 0] *= F32(2.0 ** -100)
    q[3, 0] = F32(2.0 ** -130)
    q = ref.bf16(q)
    b = batch_of(torch, tl, [5, 5], [300, 300], f.table)
    out = tl.kv_attn(to_dev(torch, q, True), f.cache, b, 0.09)
    assert np.isfinite(host(out)).all()
    keep = host(out).astype(np.float64)
    k, v = f.kv(0)
    for t in (0, 2, 3, 4):
        want, mag, top = ref.attention(q[t:t + 1].astype(np.float64), k, v, 295 + t, 0.09)
        assert np.all(np.abs(keep[t:t + 1] - want) <= ref.attention_bound(want, mag, top, 128)), t
    with np.errstate(over="ignore"):  # the huge row is a hard choice of one key
        s = k[:297, 0] @ q[1, 0].astype(np.float64)
    assert np.all(np.abs(keep[1, 0] - v[int(np.argmax(s)), 0]) <= 2.0 ** -8 * np.abs(v[int(np.argmax(s)), 0]))
    q[7, 1, 5] = np.nan
    nan = host(tl.kv_attn(to_dev(torch, q, True), f.cache, b, 0.09))
    assert np.isnan(nan[7, 1]).all()
    nan[7, 1], keep[7, 1] = 0, 0
    assert np.array_equal(nan, keep.astype(F32))
    f.cache.k_scale[int(f.table[1][4])] = float("nan")  # keys 256..299 of the second sequence
    q[7, 1, 5] = 0
    nan = host(tl.kv_attn(to_dev(torch, q, True), f.cache, b, 0.09))
    assert np.isnan(nan[5:]).all() and np.array_equal(nan[:5], keep[:5].astype(F32))


def test_attention_strided_queries_and_large_tables(torch, tl):
    """q inside a wider matrix, and a page whose codes lie past 4 GiB."""
    d, heads = 256, 8
    pages = (1 << 32) // (heads * 64 * d) + 40
    cache = tl.KVCache(torch.empty((pages, heads, 64, d), dtype=torch.int8, device="cuda:0"),
                       torch.empty((pages, heads, d, 64), dtype=torch.int8, device="cuda:0"),
                       torch.full((pages, heads), float("nan"), device="cuda:0"),
                       torch.full((pages, heads), float("nan"), device="cuda:0"))
    rng = np.random.default_rng(12)
    n = 150
    table = np.array([[pages - 1, 3, pages - 2, 0]], np.int32)
    k, v = (rng.standard_normal((n, heads, d)).astype(F32) for _ in range(2))
    tl.kv_append(cache, batch_of(torch, tl, [n], [n], table), to_dev(torch, k), to_dev(torch, v))
    model = ref.Cache(4, heads, d)  # the same pages under small names
    small = [0, 1, 2]
    model.append(small, 0, k, v)
    wide = ref.bf16(rng.standard_normal((2, 2 * heads * d + 64)).astype(F32))
    b = batch_of(torch, tl, [2], [n], table)
    q = to_dev(torch, wide, True)[:, 64:].unflatten(1, (2 * heads, d))
    out = host(tl.kv_attn(q, cache, b, 1 / 16)).astype(np.float64)
    kk, vv = (model.values(w, small, 0, n) for w in (0, 1))
    want, mag, top = ref.attention(wide[:, 64:].reshape(2, 2 * heads, d).astype(np.float64), kk, vv, n - 2, 1 / 16)
    assert np.all(np.abs(out - want) <= ref.attention_bound(want, mag, top, d))


# ---------------------------------------------------------- streams, graphs


def test_side_stream_and_graph(torch, tl):
    """The block's calls on another stream, and captured: a graph's replays
    follow the batch's arrays (one more token each) and equal the eager calls."""
    rng = np.random.default_rng(21)
    d, heads, group, K = 128, 2, 3, 256
    hq = heads * group
    steps, start = 5, 61
    table = to_dev(torch, np.array([[3, 1], [0, 2]], np.int32))
    x = to_dev(torch, outliers(rng, (steps, 2, (hq + 2 * heads) * d)))
    turn = tl.Rope.make(100, d // 2, 1e4, sections=(16, 24, 24), interleaved=True, device="cuda:0")
    qb = to_dev(torch, np.array([0, 1, 2], np.int32))
    ctx = outliers(rng, (2 * start, 2 * heads, d))

    def fresh():
        cache = tl.KVCache.empty(4, heads, d, "cuda:0")
        b = batch_of(torch, tl, [start, start], [start, start], host(table))
        c = to_dev(torch, ctx)
        tl.kv_append(cache, b, c[:, :heads], c[:, heads:])
        kv = to_dev(torch, np.array([start, start], np.int32))
        return cache, kv, tl.KVBatch(qb, kv, table, 1, 128)

    def step(cache, batch, cur, pos, stream=None):
        m = cur.unflatten(1, (hq + 2 * heads, d))
        q = tl.kv_append(cache, batch, m[:, hq:hq + heads], m[:, hq + heads:], q=m[:, :hq], rope=turn, positions=pos,
                         stream=stream)
        return tl.kv_attn(q, cache, batch, d ** -0.5, stream=stream)

    cache, kv, batch = fresh()
    pos = torch.zeros((3, 2), dtype=torch.int32, device="cuda:0")
    eager = []
    for i in range(steps):
        kv += 1
        pos += 1
        eager.append(step(cache, batch, x[i], pos).clone())
    state = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]

    side = torch.cuda.Stream()
    cache, kv, batch = fresh()
    pos.zero_()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(steps):
        with torch.cuda.stream(side):
            kv += 1
            pos += 1
        out = step(cache, batch, x[i], pos, stream=side)
        side.synchronize()
        assert torch.equal(out, eager[i])

    cache, kv, batch = fresh()
    pos.zero_()
    cur = torch.empty_like(x[0])
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache, batch, cur, pos)
    for i in range(steps):
        kv += 1
        pos += 1
        cur.copy_(x[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i]), i
    for a, b in zip(state, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ refusals


def test_refusals(torch, tl):
    cache = tl.KVCache.empty(4, 2, 64, "cuda:0")
    qb, kv = torch.tensor([0, 1], dtype=torch.int32, device="cuda:0"), torch.tensor([9], dtype=torch.int32, device="cuda:0")
    table = torch.zeros((1, 2), dtype=torch.int32, device="cuda:0")
    b = tl.KVBatch(qb, kv, table, 1, 128)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda:0")
    k = torch.zeros((1, 2, 64), device="cuda:0")
    x, w = torch.zeros((2, 64), device="cuda:0"), torch.ones(64, device="cuda:0")
    cases = [
        (TypeError, lambda: tl.rmsnorm(x.half(), w)),
        (ValueError, lambda: tl.rmsnorm(x, w[:32])),
        (tl.TernError, lambda: tl.rmsnorm(x[:, :40].contiguous(), w[:40].contiguous())),
        (ValueError, lambda: tl.rmsnorm(x.t().contiguous().t(), w)),
        (TypeError, lambda: tl.rmsnorm(x, w, residual=x, residual_out=x.bfloat16())),
        (ValueError, lambda: tl.rmsnorm(x, w, residual_out=x)),
        (TypeError, lambda: tl.rmsnorm(x, w, y=x)),
        (tl.TernError, lambda: tl.rmsnorm(x, w, eps=-1.0)),
        (TypeError, lambda: tl.KVCache(cache.k.float(), cache.v, cache.k_scale, cache.v_scale)),
        (ValueError, lambda: tl.KVCache(cache.k, cache.v[:3], cache.k_scale, cache.v_scale)),
        (ValueError, lambda: tl.KVBatch(qb, qb, table, 1, 64)),
        (TypeError, lambda: tl.KVBatch(qb, kv.long(), table, 1, 64)),
        (tl.TernError, lambda: tl.kv_attn(q, cache, tl.KVBatch(qb, kv, table, 1, 129), 1.0)),
        (tl.TernError, lambda: tl.kv_attn(q, cache, tl.KVBatch(qb, kv, table, 0, 128), 1.0)),
        (tl.TernError, lambda: tl.kv_attn(q[:, :3], cache, b, 1.0)),
        (ValueError, lambda: tl.kv_attn(q[:, :, :32], cache, b, 1.0)),
        (TypeError, lambda: tl.kv_attn(q.float(), cache, b, 1.0)),
        (tl.TernError, lambda: tl.kv_attn(q, cache, b, 0.0)),
        (tl.TernError, lambda: tl.kv_attn(q, cache, b, float("nan"))),
        (tl.TernError, lambda: tl.kv_attn(q, cache, b, 1.0, window=-1)),
        (ValueError, lambda: tl.kv_attn(q, cache, b, 1.0, out=q[:, :2])),
        (TypeError, lambda: tl.kv_append(cache, b, k, k.bfloat16())),
        (TypeError, lambda: tl.kv_append(cache, b, k, k, q=q)),
        (ValueError, lambda: tl.kv_append(cache, b, k, k[:, :1])),
        (ValueError, lambda: tl.kv_append(cache, b, k, k, rope=tl.Rope.make(8, 32, device="cuda:0"))),
        (tl.TernError, lambda: tl.kv_append(cache, b, k, k, rope=tl.Rope.make(8, 34, device="cuda:0"), positions=kv)),
        (tl.TernError, lambda: tl.kv_append(cache, b, k, k, rope=tl.Rope.make(8, 36, device="cuda:0"), positions=kv)),
        (ValueError, lambda: tl.kv_read(cache, b, 1, k_out=q)),
        (ValueError, lambda: tl.Rope.make(8, 32, sections=(8, 8, 8))),
    ]
    for i, (kind, call) in enumerate(cases):
        with pytest.raises(kind):
            call()
            raise AssertionError(f"case {i} was accepted")
    long = tl.KVBatch(qb, kv, torch.zeros((1, 4096), dtype=torch.int32, device="cuda:0"), 1, 1 << 18)
    need = tl.kv_attn_workspace_bytes(cache, long, 1, 4)
    assert need > 0
    with pytest.raises(tl.TernError, match="workspace"):
        tl.kv_attn(q, cache, long, 1.0, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda:0"))
