"""The recurrent block's operators together, as examples/decoder_block.py runs
them: chunks of a prompt, short batches and single tokens of two sequences
through norm, projection, convolution, scan, gated norm, output projection and
the norm behind it. Every stage is checked against its plain reference on what
the stage before it returned."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest

from tests import decoder_ref as dref
from tests import recurrent_ref as ref
from tests.test_gpu_decoder import operand_order
from tests.test_gpu_recurrent import dev, host, near, tl, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = ref.U


def test_block(torch, tl):  # noqa: F811
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decoder_block
    finally:
        sys.path.pop(0)
    hidden, heads, dim, groups, n_state, seqs = 512, 16, 64, 2, 128, 2
    block = decoder_block.RecurrentBlock(hidden, heads, dim, groups, n_state, seqs, seed=3)
    next_norm = torch.rand(hidden, device="cuda:0") + 0.5
    inner, ch = block.inner, block.channels
    rng = np.random.default_rng(4)
    conv, bias, a, d = (host(v).astype(np.float64) for v in (block.conv, block.conv_bias, block.a, block.d))
    for n in (70, 1, 1, 33, 4, 1, 9):  # chunks on the s8 rung, single tokens and short batches below it
        rows = seqs * n
        x = rng.standard_normal((rows, hidden)).astype(np.float32)
        stream = rng.standard_normal((rows, hidden)).astype(np.float32)
        s = dev(torch, stream)
        past, before = host(block.inputs), host(block.states)
        out, seen = block.forward(dev(torch, x), s, block.batch(n), next_norm)
        p, mixed, y, o = (host(seen[k]) for k in ("p", "mixed", "y", "o"))
        wide = isinstance(out, tuple)
        assert wide == (rows >= 17)
        for i in range(seqs):
            at = slice(i * n, (i + 1) * n)
            want, kept, e = ref.conv(p[at, inner:inner + ch].astype(np.float64), conv, bias, True, past[i])
            near(mixed[at], want, e, "conv")
            assert np.array_equal(host(block.inputs)[i], kept.astype(np.float32))
            m = mixed[at]
            r = ref.Scan(m[:, :inner].reshape(n, heads, dim), m[:, inner:inner + groups * n_state].reshape(n, groups, n_state),
                         m[:, inner + groups * n_state:].reshape(n, groups, n_state), p[at, inner + ch:inner + ch + heads], a,
                         before[i], d, host(block.dt_bias))
            near(y[at], r.y, r.y_bound(n > 8), "scan")
            assert (np.abs(host(block.states)[i] - r.s) <= r.s_bound(n > 8) + U * np.abs(r.s)).all()
        gated = ref.gated(y.reshape(rows, inner), p[:, :inner], host(block.gate_norm), 1e-6, inner // groups, True)
        if wide:
            q, scale = (host(v).astype(np.float64) for v in seen["gated"])
            step = np.abs(gated).max(1) / 127
            assert (np.abs(scale - step) <= (ref.GATED + 2 * U) * step).all()
            order = operand_order(np.tile(np.arange(64, dtype=np.int8), (1, inner // 64)))[0]  # which code lies where
            at = (np.arange(inner) // 64 * 64 + order)
            assert (np.abs(q - (gated / step[:, None])[:, at]) <= 0.5 + 127 * (2 * ref.GATED + 4 * U)).all()
        else:
            near(host(seen["gated"]), gated, ref.GATED * np.abs(gated) + 2.0 ** -100, "gated norm")
        h0 = (x + stream).astype(np.float32)
        want, e = ref.post(o, host(block.post), h0, 0.5, None, 1e-6)
        h = host(s)
        assert (np.abs(h - want) <= e).all()
        y64, _, q_ref, s_ref = dref.rmsnorm(h, host(next_norm), 1e-6)
        if wide:
            assert np.array_equal(host(out[0]), operand_order(q_ref))
            assert np.all(np.abs(host(out[1]) - s_ref) <= 32 * U * s_ref)
        else:
            near(host(out), y64, 32 * U * np.abs(y64), "next norm")


def test_example_runs(torch):  # noqa: F811
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_block.py"), "--hidden", "1280", "--prompt",
                        "300", "--chunk", "128", "--steps", "8", "--hybrid"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "309 tokens in the cache, output finite: True" in r.stdout, r.stdout
