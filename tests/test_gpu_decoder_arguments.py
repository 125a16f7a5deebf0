"""Sizes that do not fit the C calls' 32 bits are refused, not cut."""
from __future__ import annotations

import pytest

from tests.test_gpu_decoder import tl, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
WIDE = [2 ** 31, 2 ** 32 + 1, 2 ** 40 + 64, -2 ** 31 - 1]


@pytest.mark.parametrize("n", WIDE)
def test_wide_sizes(torch, tl, n):  # noqa: F811
    cache = tl.KVCache.empty(2, 1, 64, "cuda:0")
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda:0") for x in ([0, 1], [70], [[0, 1]])]
    batch = tl.KVBatch(*ints, 1, 128)
    q = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda:0")
    for call in (lambda: tl.KVBatch(*ints, n, 128), lambda: tl.KVBatch(*ints, 1, n),
                 lambda: tl.kv_attn(q, cache, batch, 1.0, window=n), lambda: tl.kv_attn(q, cache, batch, 1.0, window=64, sinks=n),
                 lambda: tl.kv_attn_workspace_bytes(cache, batch, 1, 1, n, 0),
                 lambda: tl.kv_attn_workspace_bytes(cache, batch, 1, 1, 64, n),
                 lambda: tl.kv_attn_workspace_bytes(cache, batch, n, 1), lambda: tl.kv_attn_workspace_bytes(cache, batch, 1, n)):
        with pytest.raises(ValueError):
            call()
