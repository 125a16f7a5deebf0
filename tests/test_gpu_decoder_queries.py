"""Query rows at the ends of their range: infinite elements, and rows whose
factor alone passes fp32."""
from __future__ import annotations

import pytest

from tests.test_gpu_decoder import tl, torch  # noqa: F401 (fixtures)
from tests.test_gpu_decoder_long import Random

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,lens,kernels", [(4, [300, 70], ["kv_attn"]), (40, [300, 70], ["kv_attn_tile"]),
                                            (4, [9_000, 70], ["kv_attn", "kv_attn_join"])])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("sign", [1, -1, 0])
def test_rows_of_infinite_queries_are_nan(torch, tl, n, lens, kernels, value, sign):  # noqa: F811
    """Scores are infinite of one sign (all keys share the element's sign: the
    weights are 0 / 0 or inf / inf) or of both: no row has a result. Rows beside
    them, and infinite ones that see no key, keep theirs."""
    f = Random(torch, tl, n, lens + [64], 2, 128)
    if sign:
        f.cache.k[..., 9] = sign * 7
    q = torch.randn((3 * n, 10, 128), device="cuda:0", generator=torch.Generator(device="cuda:0").manual_seed(1)).bfloat16()
    batch = tl.KVBatch(torch.arange(4, dtype=torch.int32, device="cuda:0") * n,
                       torch.tensor(lens + [0], dtype=torch.int32, device="cuda:0"), f.table, n, max(lens))
    clean = tl.kv_attn(q, f.cache, batch, 0.09)
    bad = torch.zeros((3 * n, 10), dtype=torch.bool, device="cuda:0")
    bad[1, 3] = bad[n, :] = bad[2 * n, 0] = True
    q[..., 9] = torch.where(bad, value, q[..., 9])
    out = tl.kv_attn(q, f.cache, batch, 0.09)
    assert tl.last_kernels() == kernels
    sees = bad.clone()
    sees[2 * n:] = False
    assert torch.isnan(out[sees]).all()
    assert torch.equal(out[~sees], clean[~sees])

@pytest.mark.parametrize("n", [1, 40])
def test_pages_of_zero_keys_under_a_factor_past_fp32(torch, tl, n):  # noqa: F811
    """scale times the row's power of two is past fp32; a page of zero keys still
    has scores of zero, not 0 * inf."""
    d, lens = 64, [100]
    f = Random(torch, tl, 3, lens, 1, d)
    f.cache.k.zero_()
    f.cache.k_scale.zero_()
    q = torch.full((n, 2, d), 3e38, device="cuda:0").bfloat16()
    out = tl.kv_attn(q, f.cache, f.batch(torch, tl, n), 8.0)
    f.check(torch, q, out, 0, n, 8.0)
