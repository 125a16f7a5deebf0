"""The gate z / (1 + exp(-z)) far from zero, in the gated norm and behind the
convolution."""
from __future__ import annotations

import numpy as np
import pytest

from tests import recurrent_ref as ref
from tests.test_gpu_recurrent import batch_of, dev, host, near, tl, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
F32 = np.float32
U = ref.U

# Up to the largest value, through the exponential's range (88.7) and the kernel's bound of its argument (126).
FAR = np.array([12.5, 20, 50, 86, 87, 87.25, 87.4, 87.75, 88, 88.5, 89, 100, 125.5, 126, 127, 200, 1e4, 1e30, 1e38], F32)
FAR = np.concatenate((FAR, -FAR, [0.0, -0.0, 1e-30, -1e-30])).astype(F32)

# (8 + |z|) U of the gate as near zero; below -87.3 the reciprocal of 1 + exp(-z) leaves the normal
# range and may be 0, where the gate is 87.4 * 2^-126 < 2^-119 at most.


def test_convolution(torch, tl):  # noqa: F811
    ch, n = 16, len(FAR)
    x = np.repeat(FAR[:, None], ch, 1)
    w = np.zeros((ch, 4), F32)
    w[:, 3] = 1
    state = torch.zeros((1, 3, ch), device="cuda:0")
    for bf16 in (False, True):
        xd = dev(torch, x, bf16)
        s = state.to(xd.dtype)
        y = host(tl.causal_conv(xd, dev(torch, w), s, batch_of(torch, tl, [0, n], [-1], [0])))
        z = host(xd).astype(np.float64)
        want = ref.silu(z)
        near(y, want, (8 + np.minimum(np.abs(z), 128)) * U * np.abs(want) + 2.0 ** -119)


@pytest.mark.parametrize("first", [True, False])
def test_gated_norm(torch, tl, first):  # noqa: F811
    rng = np.random.default_rng(5)
    K, most = 128, 200.0
    far = FAR[np.abs(FAR) <= most]
    z = rng.standard_normal((4, K + 16)).astype(F32)
    z[0, 8:8 + len(far)] = far
    z[1, 8:8 + K] = -rng.uniform(80, 95, K)  # every gate near the end of the range
    z[2, 8:8 + K] = -150
    x, w = rng.standard_normal((4, K)).astype(F32), rng.uniform(0.5, 1.5, K).astype(F32)
    zs = z[:, 8:8 + K].astype(np.float64)
    want = ref.gated(x, zs, w, 1e-6, 64, first)
    y = host(tl.rmsnorm_gated(dev(torch, x), dev(torch, z)[:, 8:8 + K], dev(torch, w), 1e-6, group=64, gate_first=first))
    # GATED holds for |z| < 12: two more roundings for each further |z| / 2 of the gate itself, and of
    # the sum of squares; what the gate loses is multiplied by w x rho, below 8 * 1e3
    e = (ref.GATED + 4 * np.abs(zs).max(1, keepdims=True) * U) * np.abs(want) + 2.0 ** -119 * 8e3
    near(y, want, e)
    assert (np.abs(y[2]) <= 2.0 ** -100).all()
