"""Page scales at the ends of their range: infinite and NaN ones beside rows
that do not see the page, value scales near the end of fp32."""
from __future__ import annotations

import numpy as np
import pytest

from tests import decoder_ref as ref
from tests.test_gpu_decoder import tl, torch  # noqa: F401 (fixtures)
from tests.test_gpu_decoder_long import Random, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which,bad", [(0, float("inf")), (0, float("nan")), (1, float("inf")), (1, float("nan"))])
@pytest.mark.parametrize("n,length,page,window,kernels", [
    (4, 642, 10, 0, ["kv_attn"]),                            # two rows before the page, two in it
    (40, 660, 10, 0, ["kv_attn_tile"]),
    (4, 357, 3, 100, ["kv_attn"]),                           # two rows see the page's last keys, two have left it
    (40, 370, 3, 100, ["kv_attn_tile"]),
    (4, 20_034, 313, 0, ["kv_attn", "kv_attn_join"]),
    (40, 8_980, 140, 0, ["kv_attn_tile", "kv_attn_join"]),
])
def test_scales_that_are_not_finite_stay_out_of_rows_that_do_not_see_them(torch, tl, n, length, page, window, kernels,  # noqa: F811
                                                                         which, bad):
    f = Random(torch, tl, length, [length, 300], 2, 128)
    q, clean = run(torch, tl, f, n, 10, 0.09, 3, window)
    at = int(f.table[0, page])
    (f.cache.k_scale, f.cache.v_scale)[which][at, 1] = bad
    _, out = run(torch, tl, f, n, 10, 0.09, 3, window)
    assert tl.last_kernels() == kernels
    pos = torch.arange(length - n, length, device="cuda:0")
    seen = (pos >= 64 * page) & ((pos < 64 * page + 63 + window) if window else True)
    assert seen.any() and not seen.all()
    sees = torch.zeros((2 * n, 10), dtype=torch.bool, device="cuda:0")
    sees[:n, 5:] = seen[:, None]
    assert torch.equal(torch.isnan(out).all(2), sees) and torch.equal(torch.isnan(out).any(2), sees)
    assert torch.equal(out[~sees], clean[~sees])


@pytest.mark.parametrize("n,lens,kernels", [(1, [300, 70], ["kv_attn"]), (40, [300, 70], ["kv_attn_tile"]),
                                            (1, [9_000, 70], ["kv_attn", "kv_attn_join"])])
@pytest.mark.parametrize("scale,every", [(2.0 ** 112, 1), (2.0 ** 114, 1), (2.0 ** 120, 1), (2.0 ** 113, 3)])
def test_values_up_to_the_end_of_fp32(torch, tl, n, lens, kernels, scale, every):  # noqa: F811
    """Pages of huge values, alone and among ordinary ones."""
    f = Random(torch, tl, n, lens, 2, 128)
    for s in range(2):
        f.cache.v_scale[f.table[s, :(lens[s] + 63) // 64:every].long()] = scale
    q, out = run(torch, tl, f, n, 10, 0.09, 3)
    assert tl.last_kernels() == kernels
    for s in range(2):
        f.check(torch, q, out, s, n, 0.09)


@pytest.mark.parametrize("n,heads,hq,kernels", [(1, 2, 4, ["kv_attn", "kv_attn_join"]), (40, 2, 8, ["kv_attn_tile", "kv_attn_join"]),
                                                (1, 256, 256, ["kv_attn"]), (40, 256, 256, ["kv_attn_tile"])])
def test_many_keys_of_the_least_value_scale(torch, tl, n, heads, hq, kernels):  # noqa: F811
    """The sum of weights over values of 2^-100 passes 2^113."""
    f = Random(torch, tl, n, [20_000, 17_000], heads, 64)
    f.cache.v_scale.fill_(2.0 ** -100)
    q = torch.zeros((2 * n, hq, 64), dtype=torch.bfloat16, device="cuda:0")
    out = tl.kv_attn(q, f.cache, f.batch(torch, tl, n), 0.125)
    assert tl.last_kernels() == kernels
    for s in range(2):
        f.check(torch, q, out, s, n, 0.125)


@pytest.mark.parametrize("n,lens,window,kernels", [
    (1, [600, 200], 0, ["kv_attn"]), (40, [600, 200], 150, ["kv_attn_tile"]), (4, [9_000, 300], 0, ["kv_attn", "kv_attn_join"]),
    (60, [3_000, 300], 0, ["kv_attn_tile", "kv_attn_join"])])
@pytest.mark.parametrize("scales", [(2.0 ** 120, 2.0 ** -7), (2.0 ** -7, 2.0 ** 120), (2.0 ** 118, 1.0, 2.0 ** -100),
                                    (2.0 ** -100, 2.0 ** -100, 2.0 ** -100, 2.0 ** -100, 2.0 ** 100),
                                    (2.0 ** 100, 2.0 ** -100, 2.0 ** -100, 2.0 ** -100, 2.0 ** -100)])
def test_value_scales_far_apart(torch, tl, n, lens, window, kernels, scales):  # noqa: F811
    """Keys of small values keep their weight beside keys of huge ones, in either
    order. Beside attention_bound: a weight times value scale is held in steps of
    2^-39 of the row's largest, so an element whose code is zero in every key of
    that size may lose half a step times 127 of each other key."""
    f = Random(torch, tl, 50 + n, lens, 2, 128)
    for s in range(2):
        for i in range((lens[s] + 63) // 64):
            f.cache.v_scale[int(f.table[s, i])] = scales[i % len(scales)]
    q, out = run(torch, tl, f, n, 10, 0.09, 3, window)
    assert tl.last_kernels() == kernels
    c, place = f.cache, torch.from_numpy(ref.PLACES).to("cuda:0")
    for s in range(2):
        keys = lens[s]
        pages = f.table[s, :(keys + 63) // 64].long()
        i = torch.arange(keys - n, keys, device="cuda:0")[:, None]
        j = torch.arange(keys, device="cuda:0")[None]
        hide = (j > i) | ((j <= i - window) if window else False)
        for x in range(10):
            k = (c.k[pages, x // 5].double() * c.k_scale[pages, x // 5, None, None].double()).reshape(-1, c.d)[:keys]
            w = c.v_scale[pages, x // 5].double().repeat_interleave(64)[:keys]
            v = c.v[pages, x // 5][:, :, place].transpose(1, 2).double().reshape(-1, c.d)[:keys] * w[:, None]
            raw = (q[s * n:(s + 1) * n, x].double() @ k.T * 0.09).masked_fill(hide, float("-inf"))
            p = torch.softmax(raw, 1)
            want, mag = (p @ v).cpu().numpy(), (p @ v.abs()).cpu().numpy()
            top = raw.masked_fill(hide, 0).abs().amax(1).cpu().numpy()
            step = ((~hide).sum(1) * 2.0 ** -40 * 127 * (p * w).amax(1)).cpu().numpy()[:, None]
            got = out[s * n:(s + 1) * n, x].double().cpu().numpy()
            assert np.all(np.abs(got - want) <= ref.attention_bound(want, mag, top, c.d) + step), (s, x)
