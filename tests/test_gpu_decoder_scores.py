"""Attention whose scores are large: pages of very different key scales, a
channel that all keys share, scores up to 1e30. Against torch in 64 bits, from
the codes, with the error of 32-bit scores as the bound."""
from __future__ import annotations

import math

import pytest

from tests import decoder_ref as ref
from tests.test_gpu_decoder import tl, torch  # noqa: F401 (fixtures)
from tests.test_gpu_decoder_long import Random

pytestmark = pytest.mark.gpu


def reference(torch, f, q, s, n, h, scale, window=0, sinks=0):  # noqa: F811
    """For query head h of sequence s (n rows): (out in 64 bits, bound, whether one key
    holds the row for certain).

    A score is a sum of d exact products in fp32, at worst truncated (2^-23 of
    the absolute sum each), of query elements whose bits below 2^-24 of the
    row's largest may be lost (half of that each), times a factor of four
    roundings; exponents take a few more roundings of themselves and of the
    value scale's logarithm (below 128): together E. Weights are then off by at
    most exp(2 E) of each other. The result moves by at most exp(2 E) - 1 times
    the weighted distance of the values from it, which is below 4 max|v| times
    the weight of all keys but the first. Added: 2^-11 of each probability's
    share, and the rounding to bf16."""
    c, keys = f.cache, f.lens[s]
    pages = f.table[s, :(keys + 63) // 64].long()
    place = torch.from_numpy(ref.PLACES).to("cuda:0")
    kv = h // (q.shape[1] // c.heads)
    k = (c.k[pages, kv].double() * c.k_scale[pages, kv, None, None].double()).reshape(-1, c.d)[:keys]
    v = c.v[pages, kv][:, :, place].transpose(1, 2).double() * c.v_scale[pages, kv, None, None].double()
    v = v.reshape(-1, c.d)[:keys]
    x = q[s * n:(s + 1) * n, h].double()
    i = torch.arange(keys - n, keys, device="cuda:0")[:, None]
    j = torch.arange(keys, device="cuda:0")[None]
    hide = j > i
    if window:
        hide = hide | ((j <= i - window) & (j >= sinks))
    score = (x @ k.T * scale).masked_fill(hide, -math.inf)
    size = (x.abs() @ k.abs().T * scale).masked_fill(hide, 0)
    lost = (x.abs().amax(1, keepdim=True) * k.abs().sum(1)[None] * scale).masked_fill(hide, 0)
    E = (c.d * 2.0 ** -23 * size + 2.0 ** -25 * lost + 8 * 2.0 ** -24 * (size + 128)).amax(1) + 1e-4
    p = torch.softmax(score, 1)
    out, mag = p @ v, p @ v.abs()
    first = score.argmax(1, keepdim=True)
    rest = torch.logsumexp(score.scatter(1, first, -math.inf), 1) - torch.logsumexp(score, 1)
    far = 4 * torch.exp((2 * E + torch.log(-torch.expm1(-2 * E)) + rest).clamp(max=10))  # 4 (exp(2 E) - 1) exp(rest)
    e = far.clamp(max=2)[:, None] * v.abs().max() + 2.0 ** -11 * mag
    half = 2.0 ** (torch.floor(torch.log2((out.abs() + e).clamp(min=2.0 ** -126))) - 8)
    return out, e + half, far < 1e-3


FORMS = [
    # d, kv heads, query heads, tokens of a sequence, lengths, window, sinks, kernels
    (64, 2, 8, 1, [700, 333], 0, 0, ["kv_attn"]),
    (128, 1, 5, 4, [1000, 257], 0, 0, ["kv_attn"]),
    (256, 1, 6, 1, [640, 100], 200, 4, ["kv_attn"]),
    (64, 2, 8, 1, [30_000, 1_111], 0, 0, ["kv_attn", "kv_attn_join"]),
    (128, 1, 5, 4, [20_000, 64], 0, 0, ["kv_attn", "kv_attn_join"]),
    (128, 1, 5, 40, [333, 200], 0, 0, ["kv_attn_tile"]),
    (128, 1, 5, 40, [333, 1_000], 0, 0, ["kv_attn_tile", "kv_attn_join"]),
    (64, 2, 2, 200, [513, 200], 100, 3, ["kv_attn_tile"]),
    (256, 1, 2, 100, [700, 300], 0, 0, ["kv_attn_tile"]),
    (128, 1, 3, 100, [5_000, 700], 0, 0, ["kv_attn_tile", "kv_attn_join"]),
    (256, 2, 4, 80, [4_000, 100], 0, 0, ["kv_attn_tile", "kv_attn_join"]),
]


def spread(torch, f, seed, kind):  # noqa: F811
    """Key scales of a cache of random codes: up to 4 or 100 times apart, or a
    channel of 300 that all keys share but for 3 %, beside values of one."""
    g = torch.Generator(device="cuda:0")
    g.manual_seed(seed)
    c = f.cache
    u = torch.rand(c.k_scale.shape, device="cuda:0", generator=g)
    if kind == "channel":
        c.k.copy_(torch.randint(-1, 2, c.k.shape, device="cuda:0", generator=g))
        c.k[..., 5] = torch.randint(119, 128, c.k.shape[:3], dtype=torch.int8, device="cuda:0", generator=g)
        c.k_scale.copy_((300 + 9 * u) / 127)
    else:
        c.k_scale.copy_(0.01 * kind ** u)


@pytest.mark.parametrize("kind,size", [(4, 1e4), (4, 1e5), (100, 3e3), (100, 1e8), (4, 1e30), ("channel", 260)])
@pytest.mark.parametrize("d,heads,hq,n,lens,window,sinks,kernels", FORMS)
def test_large_scores(torch, tl, d, heads, hq, n, lens, window, sinks, kernels, kind, size):  # noqa: F811
    f = Random(torch, tl, d + n, lens, heads, d)
    spread(torch, f, n, kind)
    g = torch.Generator(device="cuda:0")
    g.manual_seed(hq)
    q = torch.randn((len(lens) * n, hq, d), device="cuda:0", generator=g)
    if kind == "channel":
        q[..., 5] = size
    else:
        q *= size / (73 * 0.01)  # scores of about `size` on the page of the least scale
    q = q.bfloat16()
    out = tl.kv_attn(q, f.cache, f.batch(torch, tl, n), d ** -0.5, window=window, sinks=sinks)
    assert tl.last_kernels() == kernels
    certain = total = 0
    for s in range(len(lens)):
        for h in range(hq):
            want, bound, sure = reference(torch, f, q, s, n, h, d ** -0.5, window, sinks)
            got = out[s * n:(s + 1) * n, h].double()
            bad = ~((got - want).abs() <= bound)
            assert not bad.any(), (s, h, int(bad.any(1).sum()), float((got - want).abs().max()))
            certain, total = certain + int(sure.sum()), total + n
    if kind != "channel":
        assert certain > total / 2  # the inputs are such that the bound tells keys apart


@pytest.mark.parametrize("n", [1, 40])
def test_steep_and_flat_rows_and_pages_together(torch, tl, n):  # noqa: F811
    """Rows of large and of ordinary scores share tiles, pages of both factors
    alternate: a row's result is the same as among its like."""
    f = Random(torch, tl, 11 + n, [900, 900], 1, 128)
    f.cache.k_scale[::2] *= 50
    g = torch.Generator(device="cuda:0")
    g.manual_seed(n)
    q = torch.randn((2 * n, 4, 128), device="cuda:0", generator=g).bfloat16()
    b = f.batch(torch, tl, n)
    flat = tl.kv_attn(q, f.cache, b, 0.05)
    mixed = q.clone()
    mixed[:, 1] *= 1000
    out = tl.kv_attn(mixed, f.cache, b, 0.05)
    assert torch.equal(out[:, [0, 2, 3]], flat[:, [0, 2, 3]])
    for s in range(2):
        want, bound, _ = reference(torch, f, mixed, s, n, 1, 0.05)
        assert ((out[s * n:(s + 1) * n, 1].double() - want).abs() <= bound).all()
