"""Attention over caches long enough for every kernel's later stretches: page
ids and scales are taken 64 at a time, runs cross sequences of any length and
sequences without tokens. Against torch in 64 bits, from the codes."""
from __future__ import annotations

import numpy as np
import pytest

from tests import decoder_ref as ref
from tests.test_gpu_decoder import Filled, batch_of, check_attention, tl, to_dev, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


class Random:
    """Random codes and scales on the GPU; page tables in random order."""

    def __init__(self, torch, tl, seed, lens, heads, d):
        g = torch.Generator(device="cuda:0")
        g.manual_seed(seed)
        needs = [(n + 63) // 64 for n in lens]
        pages = sum(needs)
        self.cache = tl.KVCache(
            torch.randint(-127, 128, (pages, heads, 64, d), dtype=torch.int8, device="cuda:0", generator=g),
            torch.randint(-127, 128, (pages, heads, d, 64), dtype=torch.int8, device="cuda:0", generator=g),
            0.005 + 0.02 * torch.rand((pages, heads), device="cuda:0", generator=g),
            0.005 + 0.02 * torch.rand((pages, heads), device="cuda:0", generator=g))
        order = torch.randperm(pages, device="cuda:0", generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(needs)), -1, dtype=torch.int32, device="cuda:0")
        at = 0
        for s, n in enumerate(needs):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.lens = lens

    def batch(self, torch, tl, n):
        q = torch.arange(len(self.lens) + 1, dtype=torch.int32, device="cuda:0") * n
        return tl.KVBatch(q, torch.tensor(self.lens, dtype=torch.int32, device="cuda:0"), self.table, n, max(self.lens))

    def check(self, torch, q, out, s, n, scale, window=0, sinks=0):
        """Every row of sequence s (n tokens of the call) within attention_bound."""
        keys, c = self.lens[s], self.cache
        pages = self.table[s, :(keys + 63) // 64].long()
        place = torch.from_numpy(ref.PLACES).to("cuda:0")
        i = torch.arange(keys - n, keys, device="cuda:0")[:, None]
        j = torch.arange(keys, device="cuda:0")[None]
        hide = j > i
        if window:
            hide = hide | ((j <= i - window) & (j >= sinks))
        group = q.shape[1] // c.heads
        for h in range(c.heads):
            k = (c.k[pages, h].double() * c.k_scale[pages, h, None, None].double()).reshape(-1, c.d)[:keys]
            v = c.v[pages, h][:, :, place].transpose(1, 2).double() * c.v_scale[pages, h, None, None].double()
            v = v.reshape(-1, c.d)[:keys]
            for x in range(h * group, (h + 1) * group):
                raw = (q[s * n:(s + 1) * n, x].double() @ k.T * scale).masked_fill(hide, float("-inf"))
                p = torch.softmax(raw, 1)
                want, mag = (p @ v).cpu().numpy(), (p @ v.abs()).cpu().numpy()
                top = raw.masked_fill(hide, 0).abs().amax(1).cpu().numpy()
                got = out[s * n:(s + 1) * n, x].double().cpu().numpy()
                assert np.all(np.abs(got - want) <= ref.attention_bound(want, mag, top, c.d)), (s, x)


def run(torch, tl, f, n, hq, scale, seed, window=0, sinks=0):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    q = torch.randn((len(f.lens) * n, hq, f.cache.d), device="cuda:0", generator=g).bfloat16()
    return q, tl.kv_attn(q, f.cache, f.batch(torch, tl, n), scale, window=window, sinks=sinks)


@pytest.mark.parametrize("d,heads,hq,n,lens,window,sinks,checked", [
    (64, 8, 16, 1, [600_001], 0, 0, [0]),              # runs of more than 256 pages, few rows
    (64, 8, 16, 1, [600_001], 580_000, 7_000, [0]),    # the same with a window and many sinks
    (256, 8, 8, 40, [130_003], 0, 0, [0]),             # two blocks of few rows of one sequence
    (256, 8, 8, 70, [130_003], 0, 0, [0]),             # runs of more than 62 pages, many rows
    (128, 8, 8, 40, [4_501 - i for i in range(128)], 0, 0, [0, 77]),  # a workgroup a unit, many rows
    (64, 8, 8, 1, [16_900 - 10 * i for i in range(64)], 0, 0, [1, 63]),  # a workgroup a unit, few rows
    (64, 8, 32, 5, [40_000, 3_000, 64, 17_001], 0, 0, [0, 1, 2, 3]),  # two row tiles, runs across sequences
])
def test_long(torch, tl, d, heads, hq, n, lens, window, sinks, checked):  # noqa: F811
    f = Random(torch, tl, sum(lens), lens, heads, d)
    q, out = run(torch, tl, f, n, hq, d ** -0.5, d + n, window, sinks)
    for s in checked:
        f.check(torch, q, out, s, n, d ** -0.5, window, sinks)


@pytest.mark.parametrize("group", [2, 20, 40])
def test_runs_over_sequences_without_tokens(torch, tl, group):  # noqa: F811
    """Sequences without rows, without keys, and with rows before the first key
    between others, in runs that cross them: their rows are zero, the others right."""
    rng = np.random.default_rng(group)
    lens = [700, 64, 1500, 1, 130]
    f = Filled(torch, tl, rng, lens, 1, 64)
    wide = np.full((8, 40), -1, np.int32)
    used = [0, 2, 4, 5, 7]
    for at, s in zip(used, range(5)):
        wide[at, :f.table.shape[1]] = f.table[s]
    ns = [1, 2, 1, 0, 1, 1, 3, 2]
    kv = [700, 0, 64, 500, 1500, 1, 2000 * 64, 130]  # the second has no keys; the seventh's length is past max_kv
    q = ref.bf16(rng.standard_normal((sum(ns), group, 64)).astype(np.float32))
    qb = np.concatenate(([0], np.cumsum(ns))).astype(np.int32)
    b = tl.KVBatch(to_dev(torch, qb), to_dev(torch, np.array(kv, np.int32)), to_dev(torch, wide), 3, 40 * 64)
    out = tl.kv_attn(to_dev(torch, q, True), f.cache, b, 0.125)
    assert "kv_attn_join" in tl.last_kernels()
    got = out.float().cpu().numpy()
    assert not got[qb[1]:qb[2]].any() and not got[qb[6]:qb[7]].any()
    rows = np.concatenate([np.arange(qb[a], qb[a + 1]) for a in used])
    check_attention(f, q[rows], out[torch.from_numpy(rows).to("cuda:0")], [ns[a] for a in used], 0.125)


@pytest.mark.parametrize("d,n,group,window", [(128, 200, 1, 0), (256, 60, 3, 0), (256, 7, 4, 0), (128, 1, 5, 3000)])
def test_graph_of_every_kernel(torch, tl, d, n, group, window):  # noqa: F811
    """Captured calls (operands in more than 64 KiB of LDS, runs and their join
    among them) replay with new lengths and queries as the eager calls do."""
    f = Random(torch, tl, d + n, [5_003, 640, 2_111], 2, d)
    batch = f.batch(torch, tl, n)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(5)
    qs = [torch.randn((3 * n, 2 * group, d), device="cuda:0", generator=g).bfloat16() for _ in range(4)]
    lens = [[5_003, 640, 2_111], [4_100, 600, 64 + n], [n, 321, 2_000], [5_000, 639, 1_999]]
    ws = tl.kv_attn_workspace(f.cache, batch, 3 * n, 2 * group, window, 2)

    def call(q):
        return tl.kv_attn(q, f.cache, batch, d ** -0.5, window=window, sinks=2, workspace=ws)

    def at(i):
        batch.kv_len.copy_(torch.tensor(lens[i], dtype=torch.int32))

    eager = []
    for i, q in enumerate(qs):
        at(i)
        eager.append(call(q).clone())
    cur = qs[0].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = call(cur)
    for i in (1, 3, 0, 2, 1):
        at(i)
        cur.copy_(qs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i]), i
        assert torch.equal(call(qs[i]), eager[i]), i


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("which,bad", [(0, float("inf")), (0, float("nan")), (1, float("inf")), (1, float("nan"))])
def test_scales_that_are_not_finite(torch, tl, n, which, bad):  # noqa: F811
    """A page whose scale is not finite (it holds a value that was not) makes
    exactly the rows NaN that see it, of its head."""
    f = Random(torch, tl, 7, [700, 700], 2, 128)
    q, clean = run(torch, tl, f, n, 10, 0.09, 3)
    page = int(f.table[1, 10])  # keys 640 .. 699 of the second sequence
    (f.cache.k_scale, f.cache.v_scale)[which][page, 1] = bad
    _, out = run(torch, tl, f, n, 10, 0.09, 3)
    sees = torch.zeros((2 * n, 10), dtype=torch.bool, device="cuda:0")
    sees[n + max(0, 640 - (700 - n)):, 5:] = True
    assert torch.equal(torch.isnan(out).all(2), sees) and torch.equal(torch.isnan(out).any(2), sees)
    assert torch.equal(out[~sees], clean[~sees])
