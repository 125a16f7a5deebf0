"""y of prompts keeps what fp32 sums would give: weights inside a block and the
state before it enter the matrix products as two bf16 numbers each."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_gpu_recurrent import SEGMENTS, U, ScanCase, host, near, run_scan, tl, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

# The upper part is what the upper half of a float holds, off by less than 2^-7 of the value; the lower
# part is that rest rounded to bf16, off by half a step, 2^-8 of it: 2^-15 of every term of y, beside the
# recurrence and the sums in fp32 (as recurrent_ref has them).
TWO_PARTS = 2.0 ** -15


def check(c, y, i):
    r = c.reference(i)
    e = (r.rel[..., None] + (r.N + 72) * U + TWO_PARTS) * r.ymag
    got, want = y[c.begin[i]:c.begin[i + 1]], r.y
    near(got, want, e, i)
    # Where terms cancel to less than 2^-6 of their magnitudes, each result is off by less than half a step of
    # bf16, 2^-8 of it; all together, where the terms' own bound is 2^-15 of the magnitudes, by less than 2^-7.
    small = np.abs(want) < 2.0 ** -6 * r.ymag
    assert small.any()
    off = np.linalg.norm((got - want)[small])
    assert off <= 2.0 ** -8 * np.linalg.norm(want[small]) + np.linalg.norm(e[small])


@pytest.mark.parametrize("skip", [True, False])
@pytest.mark.parametrize("p,n,heads,groups,lens", [
    (64, 128, 12, 2, [200, 33]), (32, 64, 5, 1, [130]), (128, 256, 3, 1, [70]), (64, 64, 3, 1, [33, 64]), (32, 256, 4, 2, [96]),
    (128, 128, 2, 1, [95])])
def test_prompts(torch, tl, p, n, heads, groups, lens, skip):  # noqa: F811
    c = ScanCase(torch, 5 * p + n + heads, lens, heads, groups, p, n, skip=skip)
    y, _ = run_scan(torch, tl, c)
    assert tl.last_kernels() == ["scan_prepare", "scan_blocks"]
    for i in range(len(lens)):
        check(c, host(y), i)


@pytest.mark.parametrize("p,n", [(64, 128), (128, 64)])
def test_segments(torch, tl, p, n):  # noqa: F811
    c = ScanCase(torch, 31, [1500], 2, 1, p, n, skip=False)
    y, _ = run_scan(torch, tl, c)
    assert sorted(tl.last_kernels()) == SEGMENTS
    check(c, host(y), 0)
