"""Plain references of the decoder operators (norm, cache, attention), numpy on
the CPU, from the definitions in tern.h: integers by the stated fp32 steps,
everything else in 64 bits. They share no code with the library."""
from __future__ import annotations

import numpy as np

PAGE = 64
F32 = np.float32


def v_place(slot):
    """Place of a token slot inside a row of v."""
    tile, rest = divmod(slot, 16)
    return 16 * (rest // 4) + 4 * tile + rest % 4


PLACES = np.array([v_place(s) for s in range(PAGE)])


def bf16(x):
    """float32 values rounded to nearest even bf16 (finite input), as float32."""
    b = np.ascontiguousarray(x, F32).view(np.uint32).astype(np.uint64)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32)).view(F32)


def half_ulp(x):
    """Largest error of rounding |x| to bf16 (8 significant bits; subnormals from 2^-126 down)."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -126)))
    return 2.0 ** (e - 8)


def codes(v, a):
    """clamp(rne(fl(v / a)), +-127) for fp32 v and scale a (a > 0), else zeros."""
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((v.astype(F32) / a.astype(F32)).astype(F32))
    return np.where(a > 0, np.clip(q, -127, 127), 0).astype(np.int8)


def rmsnorm(x, w, eps, r=None, r_bf16=False):
    """(y in 64 bits, residual, codes, scale in 64 bits) for fp32 inputs."""
    h = x.astype(F32)
    if r is not None:
        h = (h + r.astype(F32)).astype(F32)
        if r_bf16:
            h = bf16(h)
    v = (h * w.astype(F32)).astype(F32)
    rho = 1.0 / np.sqrt((h.astype(np.float64) ** 2).mean(1) + eps)
    a = (np.abs(v).max(1) / F32(127)).astype(F32)
    return v.astype(np.float64) * rho[:, None], h, codes(v, a[:, None]), rho * a.astype(np.float64)


class Cache:
    """The cache on the host: codes by (page, head, slot, element) and scales."""

    def __init__(self, pages, heads, d):
        self.pages, self.heads, self.d = pages, heads, d
        self.c = [np.zeros((pages, heads, PAGE, d), np.int8) for _ in range(2)]
        self.s = [np.zeros((pages, heads), F32) for _ in range(2)]

    def append(self, table, start, k, v):
        """k, v: fp32 [n, heads, d], the tokens start .. start + n - 1 of a sequence."""
        n = k.shape[0]
        for which, x in enumerate((k, v)):
            for p in range(start // PAGE, (start + n - 1) // PAGE + 1):
                lo, hi, page = max(start, p * PAGE), min(start + n, (p + 1) * PAGE), table[p]
                new = x[lo - start:hi - start].transpose(1, 0, 2)
                a = (np.abs(new).max((1, 2)) / F32(127)).astype(F32)
                if lo > p * PAGE:
                    old = self.s[which][page].copy()
                    a = np.maximum(a, old)
                    held = self.c[which][page][:, :lo - p * PAGE]
                    grown = codes((held.astype(F32) * old[:, None, None]).astype(F32), a[:, None, None])
                    held[...] = np.where((a > old)[:, None, None], grown, held)
                self.s[which][page] = a
                self.c[which][page][:, lo - p * PAGE:hi - p * PAGE] = codes(new, a[:, None, None])

    def values(self, which, table, first, last):
        """[last - first, heads, d] in 64 bits."""
        t = np.arange(first, last)
        pages = np.asarray(table)[t // PAGE]
        return self.c[which][pages, :, t % PAGE].astype(np.float64) * self.s[which][pages].astype(np.float64)[..., None]


def rope(x, table, axis, positions):
    """x fp32 [tokens, heads, d] turned: every product and sum rounded to fp32."""
    pairs = table.shape[1]
    pos = np.clip(positions[np.minimum(axis, positions.shape[0] - 1)], 0, table.shape[0] - 1)  # [pairs, tokens]
    cs = table[pos, np.arange(pairs)[:, None]].transpose(1, 0, 2)[:, None]  # [tokens, 1, pairs, 2]
    a, b = x[..., :pairs].astype(F32), x[..., pairs:2 * pairs].astype(F32)
    c, s = cs[..., 0].astype(F32), cs[..., 1].astype(F32)
    return np.concatenate((a * c - b * s, b * c + a * s, x[..., 2 * pairs:]), -1).astype(F32)


def visible(i, keys, window, sinks):
    j = np.arange(keys)
    see = j <= i
    if window:
        see &= (j > i - window) | (j < sinks)
    return see


def attention(q, k, v, first, scale, window=0, sinks=0, present=None):
    """q [n, q_heads, d] standing at first .. first + n - 1; k, v [keys, heads,
    d]; all in 64 bits. Returns (out, the probability-weighted mean of |v|, the
    largest |score| of each row [n, q_heads])."""
    n, hq, d = q.shape
    keys, heads = k.shape[:2]
    out, mag, top = np.zeros((n, hq, d)), np.zeros((n, hq, d)), np.zeros((n, hq))
    for t in range(n):
        see = visible(first + t, keys, window, sinks)
        if present is not None:
            see &= present
        if not see.any():
            continue
        for h in range(hq):
            kh = h // (hq // heads)
            s = scale * (k[see, kh] @ q[t, h])
            p = np.exp(s - s.max())
            out[t, h] = p @ v[see, kh] / p.sum()
            mag[t, h] = p @ np.abs(v[see, kh]) / p.sum()
            top[t, h] = np.abs(s).max()
    return out, mag, top


def attention_bound(out, mag, top, d):
    """How far the kernel's bf16 output may be from `out`: its own rounding; the rounding of each probability to fp16 (2^-11) and the
    fp32 error of its exponent (the product's d roundings and a few more,
    2^-24 each, of the largest score in powers of two, in the numerator and in
    the sum), each on the weighted mean of |v|."""
    e = (2.0 ** -11 + 2 * (d + 16) * 2.0 ** -24 * (top[..., None] * 1.5 + 1)) * mag
    return half_ulp(np.abs(out) + e) + e
