"""A draft that is rejected: kv_len goes back, later appends overwrite its
slots, but what it did to the tokens on its page stays."""
from __future__ import annotations

import numpy as np
import pytest

from tests import decoder_ref as ref
from tests.test_gpu_decoder import batch_of, check_cache, host, tl, to_dev, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def test_a_rejected_draft_coarsens_the_tokens_of_its_page(torch, tl):  # noqa: F811
    """Tokens of size one, a draft of size fifty on the same page, rejected, then
    tokens of size one again: the page's scale stays grown, and its tokens are
    off by up to a half of it beyond their own half code; the page before and the
    page after are as without the draft."""
    rng = np.random.default_rng(6)
    heads, d = 2, 64
    table = np.array([[3, 1, 0]], np.int32)
    old, draft, new = (rng.standard_normal((n, heads, d)).astype(np.float32) for n in (100, 4, 60))
    draft *= np.float32(50)
    caches, models = [], []
    for drafted in (False, True):
        cache, model = tl.KVCache.empty(4, heads, d, "cuda:0"), ref.Cache(4, heads, d)
        steps = [(old, 0)] + ([(draft, 100)] if drafted else []) + [(new, 100)]
        for x, start in steps:
            n = len(x)
            tl.kv_append(cache, batch_of(torch, tl, [n], [start + n], table, max_q=n, max_kv=192), to_dev(torch, x),
                         to_dev(torch, x))
            model.append(table[0], start, x, x)
        check_cache(cache, model, table, [160])
        caches.append(cache)
        models.append(model)
    x = np.concatenate((old, new))
    for p in (0, 2):
        assert torch.equal(caches[0].k_scale[table[0, p]], caches[1].k_scale[table[0, p]])
    for which in (0, 1):
        for drafted, model in enumerate(models):
            got = model.values(which, table[0], 0, 160)
            scale = np.repeat(model.s[which][table[0]], 64, axis=0)[:160, :, None].astype(np.float64)
            # half a code of the scale a token came with and half of the one its page
            # grew to, both at most the last scale, and fp32's own roundings
            assert np.all(np.abs(got - x) <= 1.0001 * scale)
            # scales: about 3.5 / 127 without the draft, 50 times that with it
            assert (np.abs(got - x)[64:128].max() > 0.1) == bool(drafted)
    # the page of the draft: its scale is the draft's
    grown = np.abs(draft).max((0, 2)) / np.float32(127)
    assert np.array_equal(models[1].s[0][table[0, 1]], grown.astype(np.float32))


@pytest.mark.parametrize("value", [np.inf, np.nan])
def test_a_rejected_draft_that_is_not_finite_loses_the_tokens_of_its_page(torch, tl, value):  # noqa: F811
    """Their codes become 0 or -127 under a scale that is not finite: a caller
    that may take a draft back copies the page it begins in."""
    rng = np.random.default_rng(7)
    heads, d = 2, 64
    table = np.array([[1, 0]], np.int32)
    old = rng.standard_normal((100, heads, d)).astype(np.float32)
    draft = rng.standard_normal((2, heads, d)).astype(np.float32)
    draft[0, 1, 5] = value
    cache = tl.KVCache.empty(2, heads, d, "cuda:0")

    def append(x, start):
        tl.kv_append(cache, batch_of(torch, tl, [len(x)], [start + len(x)], table, max_q=100, max_kv=128), to_dev(torch, x),
                     to_dev(torch, x))

    def read():
        k, v = tl.kv_read(cache, batch_of(torch, tl, [100], [100], table, max_q=100, max_kv=128), 100)
        return host(k), host(v)

    append(old, 0)
    clean = read()
    kept = [t[0].clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]  # page 0 holds tokens 64 ..
    append(draft, 100)
    for got, was in zip(read(), clean):
        assert not np.isfinite(got[64:, 1]).any()
        assert np.array_equal(got[:64], was[:64])
    for t, saved in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), kept):
        t[0] = saved
    for got, was in zip(read(), clean):
        assert np.array_equal(got, was)
