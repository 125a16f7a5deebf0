"""The operators together, as examples/decoder_block.py runs them: chunks of a
prompt and single tokens of two sequences through norm, projection, rotary
append, attention and output projection. Every stage is checked against its
plain reference on what the stage before it returned."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest

from tests import decoder_ref as ref
from tests.test_gpu_decoder import check_cache, host, operand_order, tl, to_dev, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block(torch, tl):  # noqa: F811
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decoder_block
    finally:
        sys.path.pop(0)
    hidden, hq, hkv, d, seqs, most = 512, 6, 2, 128, 2, 192
    block = decoder_block.DecoderBlock(hidden, hq, hkv, d, seqs, most, seed=3, sections=(16, 24, 24))
    rng = np.random.default_rng(4)
    model = ref.Cache(block.cache.pages, hkv, d)
    table, rope, axis = host(block.table), host(block.rope.table), host(block.rope.axis)
    stream = np.zeros((0, 0), np.float32)
    length = 0
    for n in (70, 1, 1, 33, 4, 1):  # chunks on the s8 rung, single tokens and a short batch below it
        rows = seqs * n
        x = rng.standard_normal((rows, hidden)).astype(np.float32)
        stream = rng.standard_normal((rows, hidden)).astype(np.float32)
        positions = rng.integers(0, most, (3, rows)).astype(np.int32)
        block.kv_len += n
        length += n
        s = to_dev(torch, stream)
        y, seen = block.forward(to_dev(torch, x), s, to_dev(torch, positions), block.batch(n))
        # norm
        y64, h, q_ref, s_ref = ref.rmsnorm(x, host(block.norm), 1e-6, stream)
        assert np.array_equal(host(s), h)
        if isinstance(seen["normed"], tuple):
            assert np.array_equal(host(seen["normed"][0]), operand_order(q_ref))
            assert np.all(np.abs(host(seen["normed"][1]) - s_ref) <= 32 * 2.0 ** -24 * s_ref)
        else:
            e = 32 * 2.0 ** -24 * np.abs(y64)
            assert np.all(np.abs(host(seen["normed"]) - y64) <= ref.half_ulp(np.abs(y64) + e) + e)
        # append
        heads = host(seen["qkv"]).reshape(rows, hq + 2 * hkv, d)
        turned = ref.rope(heads[:, :hq + hkv], rope, axis, positions)
        assert np.array_equal(host(seen["q"]), ref.bf16(turned[:, :hq]))
        for i in range(seqs):
            at = slice(i * n, (i + 1) * n)
            model.append(table[i], length - n, turned[at, hq:], heads[at, hq + hkv:])
        check_cache(block.cache, model, table, [length] * seqs)
        # attention
        q, o = host(seen["q"]).astype(np.float64), host(seen["o"]).astype(np.float64)
        for i in range(seqs):
            at = slice(i * n, (i + 1) * n)
            k, v = (model.values(w, table[i], 0, length) for w in (0, 1))
            want, mag, top = ref.attention(q[at], k, v, length - n, d ** -0.5)
            assert np.all(np.abs(o[at] - want) <= ref.attention_bound(want, mag, top, d))
        assert y.shape == (rows, hidden) and torch.isfinite(y).all()


def test_example_runs(torch):  # noqa: F811
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_block.py"), "--hidden", "1280", "--prompt",
                        "300", "--chunk", "128", "--steps", "8"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "309 tokens in the cache, output finite: True" in r.stdout, r.stdout
