"""Plain references of the recurrent block's operators (convolution, scan, gated
norm, norm behind a block), numpy on the CPU in 64 bits from the definitions in
tern.h, and how far the kernels may be from them. They share no code with the
library."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1 + np.exp(-z))


def conv(x, w, bias, act, past):
    """x [n, ch], past [width - 1, ch]. Returns (y, the inputs the state keeps, a bound of y's error in fp32)."""
    k = w.shape[1]
    rows = np.concatenate((past, x)).astype(np.float64)
    n = x.shape[0]
    terms = [rows[j:j + n] * w[:, j] for j in range(k)]
    y = sum(terms) + (0 if bias is None else bias)
    # at most `width` products and sums after the bias, each rounded once
    e = k * U * (sum(np.abs(t) for t in terms) + (0 if bias is None else np.abs(bias)))
    if act:
        # |d silu / dz| < 1.1; log2(e) rounded, the exponential (2 ulp) and its correction,
        # sum, reciprocal (1 ulp), product
        y, e = silu(y), 1.1 * e + (8 + np.abs(y)) * U * np.abs(silu(y)) + 2.0 ** -120
    return y, rows[rows.shape[0] - (k - 1):], e


class Scan:
    """y and S of one sequence with the sums of magnitudes behind them, which
    bound the kernels' rounding errors."""

    def __init__(self, x, b, c, dt, a, state, d=None, dt_bias=None, softplus=True):
        """x [n, heads, p], b and c [n, groups, N], dt [n, heads], state [heads, N, p]."""
        n, heads, _ = x.shape
        g = heads // b.shape[1]
        x, b, c, dt = (np.asarray(v, np.float64) for v in (x, b, c, dt))
        v = dt + (0 if dt_bias is None else np.asarray(dt_bias, np.float64))
        self.step = np.logaddexp(0, v) if softplus else v
        # fp32 errors of D: the sum's rounding and the softplus' few, relative
        self.step_error = (8 + np.abs(v)) * U if softplus else 2 * U * np.ones_like(v)
        s, mag = np.array(state, np.float64), np.abs(np.asarray(state, np.float64))
        worst = np.zeros(heads)
        self.y, self.ymag = np.zeros(x.shape), np.zeros(x.shape)
        self.rel = np.zeros((n, heads))  # of the recurrence: relative to the magnitudes
        for t in range(n):
            D = self.step[t]
            keep = np.exp(D * a)
            # exponential: 4 ulp and the error of D a; two products and a sum for the update
            worst = worst + 12 * U + (np.abs(D * a) + 1) * (self.step_error[t] + 2 * U)
            u = (D[:, None] * x[t])[:, None, :]
            bt, ct = (np.repeat(m[t], g, 0)[:, :, None] for m in (b, c))
            s = keep[:, None, None] * s + bt * u
            mag = keep[:, None, None] * mag + np.abs(bt * u)
            skip = 0 if d is None else d[:, None] * x[t]
            self.y[t] = (ct * s).sum(1) + skip
            self.ymag[t] = (np.abs(ct) * mag).sum(1) + np.abs(skip)
            self.rel[t] = worst
        self.s, self.smag = s, mag
        self.N = state.shape[1]

    # Token by token: the recurrence's errors, and for y a sum of N + 1 terms
    # (N / 4 products one after the other, then a tree). In blocks: sums of up to N +
    # 64 products; a term of y has one factor rounded to bf16 (of the block's weights or
    # of the state before it), off by at most 2^-8 of itself. The state's terms keep 24 bits.
    def y_bound(self, blocks):
        e = self.rel[..., None] + (self.N + 8) * U + (2.0 ** -8 + 64 * U if blocks else 0)
        return e * self.ymag

    def s_bound(self, blocks):
        e = (self.rel[-1] if len(self.rel) else np.zeros(self.s.shape[0]))[:, None, None]
        return (e + (64 * U if blocks else 0)) * self.smag


def gated(x, z, w, eps, group, first):
    """v of tern_rmsnorm_gated, [T, K]."""
    x, z, w = (np.asarray(m, np.float64) for m in (x, z, w))
    g = silu(z)
    u = (x * g if first else x).reshape(x.shape[0], -1, group)
    with np.errstate(divide="ignore", invalid="ignore"):
        rho = 1 / np.sqrt((u * u).mean(2, keepdims=True) + eps)
        v = (u * np.where(np.isinf(rho), 0, rho)).reshape(x.shape) * w
    return v if first else v * g


# The gated norm's relative error for |z| < 12: the gate 8 + |z|, four products; the
# sum of squares twice that of the operands and up to 16 + 32 + 6 sums one after the
# other, halved by the root; root, quotient.
GATED = 84 * U


def post(x, pw, r, scale, gate, eps):
    """(h before its rounding, bound of its fp32 error)."""
    x, pw, r = (np.asarray(m, np.float64) for m in (x, pw, r))
    with np.errstate(divide="ignore", invalid="ignore"):
        rho = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    p = scale * (1 if gate is None else np.asarray(gate, np.float64)) * x * pw * np.where(np.isinf(rho), 0, rho)
    # 32 ulp for the norm as in the plain norm, three products, a sum
    return r + p, 36 * U * np.abs(p) + U * (np.abs(r) + np.abs(p))
