"""The norm of tokens whose products with the weight are all zero, without an eps."""
from __future__ import annotations

import pytest

from tests.test_gpu_decoder import tl, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_outputs_of_a_zero_token_agree(torch, tl, eps):  # noqa: F811
    """Codes and scale are zero, and so is y: not 0 / 0."""
    x = torch.randn((4, 256), device="cuda:0")
    x[1] = 0
    x[2] = -0.0
    w = torch.ones(256, device="cuda:0")
    y = torch.full((4, 256), 7.0, dtype=torch.bfloat16, device="cuda:0")
    q, s = tl.rmsnorm_s8(x, w, eps, y=y)
    assert not q[1:3].any() and not s[1:3].any()
    assert not y[1:3].any()
    assert torch.isfinite(y).all()
    assert torch.equal(tl.rmsnorm(x, w, eps), y)
    nan = x.clone()
    nan[1, 5] = float("nan")
    assert torch.isnan(tl.rmsnorm(nan, w, eps)[1]).all()
