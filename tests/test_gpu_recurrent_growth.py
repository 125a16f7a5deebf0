"""States that grow (D a > 0) through prompts cut into segments: the growth of a
segment's hundreds of rows may pass fp32 where no state does."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_gpu_recurrent import SEGMENTS, F32, ScanCase, host, run_scan, tl, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def case(torch, n, p=64, state_dim=128):  # noqa: F811
    """One sequence of two heads: the first grows by dt a row, the second hardly changes."""
    c = ScanCase(torch, 21, [n], 2, 1, p, state_dim, softplus=False)
    c.a = np.array([1, -1e-3], F32)
    c.dt[:] = 1e-3
    return c


@pytest.mark.parametrize("p,state_dim", [(64, 128), (128, 64), (32, 256)])
def test_nothing_grows_to_nothing(torch, tl, p, state_dim):  # noqa: F811
    """A state of zeros and rows of zeros stay zeros: exp(32) a block of 32 rows, segments of at least four."""
    n = 4096
    c = case(torch, n, p, state_dim)
    c.dt[:n - 50] = 1
    c.x[:n - 50] = 0
    c.src = [-1]
    y, state = run_scan(torch, tl, c)
    assert sorted(tl.last_kernels()) == SEGMENTS
    assert np.isfinite(host(y)).all() and (host(y)[:n - 50] == 0).all()
    c.check(host(y), host(state))


def test_growth_past_fp32_of_a_small_state(torch, tl):  # noqa: F811
    """A state near 1e-36 grown by exp(150) is near 1e29."""
    n = 4096
    c = case(torch, n)
    c.dt[:150] = 1
    c.x[:150] = 0
    c.pool *= F32(1e-36)
    y, state = run_scan(torch, tl, c)
    assert sorted(tl.last_kernels()) == SEGMENTS
    c.check(host(y), host(state))


def test_growth_and_decay_cancel(torch, tl):  # noqa: F811
    """Rows that grow by exp(100) and then decay by as much inside one segment: dt of both signs."""
    n = 4096
    c = case(torch, n)
    c.dt[:100] = 1
    c.dt[100:200] = -1
    c.x[:200] = 0
    c.pool *= F32(1e-12)
    y, state = run_scan(torch, tl, c)
    assert sorted(tl.last_kernels()) == SEGMENTS
    c.check(host(y), host(state))
