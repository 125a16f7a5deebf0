"""Which kernels the attention runs for the shapes of the other tests: each of
them exists for a path, named here, and the host chooses paths by rules that
may move."""
from __future__ import annotations

import pytest

from tests.test_gpu_decoder import ATTN, tl, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
FEW, TILE = ["kv_attn"], ["kv_attn_tile"]
JOIN = ["kv_attn_join"]

ATTN_KERNELS = [FEW, FEW, FEW, FEW, FEW, TILE, FEW, TILE, TILE, TILE, TILE, TILE, FEW, FEW, TILE, TILE, FEW, TILE]

# d, kv heads, query heads, tokens of a sequence, lengths, window, sinks
LONG = [
    ((64, 8, 16, 1, [600_001], 0, 0), FEW + JOIN),
    ((64, 8, 16, 1, [600_001], 580_000, 7_000), FEW + JOIN),
    ((256, 8, 8, 40, [130_003], 0, 0), FEW + JOIN),
    ((256, 8, 8, 70, [130_003], 0, 0), TILE + JOIN),
    ((128, 8, 8, 40, [4_501 - i for i in range(128)], 0, 0), TILE),
    ((64, 8, 8, 1, [16_900 - 10 * i for i in range(64)], 0, 0), FEW),
    ((64, 8, 32, 5, [40_000, 3_000, 64, 17_001], 0, 0), FEW + JOIN),
    # captured calls
    ((128, 2, 2, 200, [5_003, 640, 2_111], 0, 2), TILE + JOIN),
    ((256, 2, 6, 60, [5_003, 640, 2_111], 0, 2), TILE + JOIN),
    ((256, 2, 8, 7, [5_003, 640, 2_111], 0, 2), FEW + JOIN),
    ((128, 2, 10, 1, [5_003, 640, 2_111], 3_000, 2), FEW + JOIN),
]
SHAPES = [((d, heads, heads * group, max(ns), lens, window, sinks), kernels)
          for (d, heads, group, ns, lens, window, sinks), kernels in zip(ATTN, ATTN_KERNELS)] + LONG


def test_every_shape_is_listed():
    assert len(ATTN) == len(ATTN_KERNELS)


@pytest.mark.parametrize("shape,kernels", SHAPES)
def test_kernels_of_the_tests_shapes(torch, tl, shape, kernels):  # noqa: F811
    """No page is present, so that no cache of that length is needed: every row
    sees nothing."""
    d, heads, hq, n, lens, window, sinks = shape
    seqs = len(lens)
    cache = tl.KVCache.empty(1, heads, d, "cuda:0")
    table = torch.full((seqs, (max(lens) + 63) // 64), -1, dtype=torch.int32, device="cuda:0")
    batch = tl.KVBatch(torch.arange(seqs + 1, dtype=torch.int32, device="cuda:0") * n,
                       torch.tensor(lens, dtype=torch.int32, device="cuda:0"), table, n, max(lens))
    q = torch.ones((seqs * n, hq, d), dtype=torch.bfloat16, device="cuda:0")
    out = tl.kv_attn(q, cache, batch, d ** -0.5, window=window, sinks=sinks, out=torch.ones_like(q))
    assert tl.last_kernels() == kernels
    assert not out.any()
