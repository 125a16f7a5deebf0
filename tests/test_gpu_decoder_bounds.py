"""Batch arrays at the ends of their type: nothing is read or written for the
sequences they contradict."""
from __future__ import annotations

import pytest

from tests.test_gpu_decoder import tl, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
LEAST, MOST = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("begin", [[MOST, LEAST, 0], [MOST, MOST, LEAST], [LEAST, MOST, LEAST], [LEAST, LEAST, MOST],
                                   [MOST, LEAST + 1, MOST]])
@pytest.mark.parametrize("length", [1, 64, 100, LEAST, MOST])
def test_q_begin_whose_differences_wrap(torch, tl, begin, length):  # noqa: F811
    """A difference of two entries that wraps to a small count is no count."""
    heads, d, rows = 2, 64, 3
    cache = tl.KVCache.empty(4, heads, d, "cuda:0")
    cache.k.fill_(3)
    cache.v.fill_(5)
    cache.k_scale.fill_(1)
    cache.v_scale.fill_(1)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda:0")
    batch = tl.KVBatch(torch.tensor(begin, dtype=torch.int32, device="cuda:0"),
                       torch.full((2,), length, dtype=torch.int32, device="cuda:0"), table, 2, 128)
    x = torch.ones((rows, heads, d), device="cuda:0")
    tl.kv_append(cache, batch, x, x)
    for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
        assert torch.equal(a, b)
    k, v = (torch.full((rows, heads, d), 7.0, dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    tl.kv_read(cache, batch, rows, k_out=k, v_out=v)
    out = torch.full((rows, 2 * heads, d), 7.0, dtype=torch.bfloat16, device="cuda:0")
    tl.kv_attn(torch.ones_like(out), cache, batch, 0.1, out=out)
    for t in (k, v, out):
        assert (t == 7).all()
