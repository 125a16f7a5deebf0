"""The scan in blocks with more heads a group than one workgroup of its first
launch takes (eight), whole and partial ones, against the reference."""
from __future__ import annotations

import pytest

from tests.test_gpu_recurrent import SEGMENTS, ScanCase, host, run_scan, tl, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("p,n,heads,groups", [
    (64, 128, 9, 1), (64, 128, 40, 2), (64, 128, 160, 8), (128, 64, 11, 1), (128, 64, 24, 2), (32, 64, 17, 1), (32, 128, 27, 3),
    (32, 256, 16, 1), (128, 256, 18, 2), (64, 64, 33, 3)])
@pytest.mark.parametrize("lens", [[70], [33, 0, 9, 31]])
def test_heads_of_a_group(torch, tl, p, n, heads, groups, lens):  # noqa: F811
    c = ScanCase(torch, p + n + heads, lens, heads, groups, p, n)
    y, state = run_scan(torch, tl, c)
    assert tl.last_kernels() == ["scan_prepare", "scan_blocks"]
    c.check(host(y), host(state))


@pytest.mark.parametrize("p,n,heads,groups,lens", [(64, 128, 20, 1, [1700]), (32, 64, 26, 2, [1300, 40]), (128, 128, 9, 1, [900, 1100])])
def test_heads_of_a_group_in_segments(torch, tl, p, n, heads, groups, lens):  # noqa: F811
    c = ScanCase(torch, p + n + heads, lens, heads, groups, p, n)
    y, state = run_scan(torch, tl, c)
    assert sorted(tl.last_kernels()) == SEGMENTS
    c.check(host(y), host(state))
