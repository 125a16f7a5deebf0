"""Sizes of the recurrent block's operators at the limits of a launch, without
a GPU: what a launch cannot hold is refused before any HIP call."""
from __future__ import annotations

import pytest

from tests.test_host_recurrent import P, SHAPE, batch, conv, tl  # noqa: F401 (fixture)


@pytest.mark.parametrize("type,per", [(0, 4), (1, 8)])
def test_conv_threads_of_a_sequence_fit_31_bits(tl, type, per):  # noqa: F811
    """A thread's number within its sequence has 31 bits; max_q bounds it, however few the rows."""
    ch = 1 << 20
    runs = (1 << 31) // (ch // per)  # of 16 tokens: 2^31 threads
    for max_q in (16 * runs + 1, 16 * runs + 16, min(2 * 16 * runs - 16, 1 << 19)):
        assert conv(tl, batch(tl, seqs=1, max_q=max_q), rows=32, type=type, ch=ch, xs=ch, ys=ch) == SHAPE, max_q
        assert b"too large" in tl.lib().tern_last_error()
