"""The 8-bit serving operators in float64: the int8 quantizer, the linear layer
on int8 codes, the paged 8-bit key/value cache and attention over it.

The quantizer's codes are fixed by its float32 arithmetic (``scale = amax / 127``,
``inverse = 1 / scale``, ``code = rint(x * inverse)``, each operation rounded to
float32), so ``quantize_ref`` does those steps in float32 and everything built on
the codes is float64.
"""
from __future__ import annotations

import numpy as np

F32 = np.float32
TINY = F32(2.0 ** -126)


def scale_ref(amax) -> np.float32:
    amax = F32(amax)
    if not np.isfinite(amax):
        return F32(np.nan)
    s = amax / F32(127)
    return F32(0) if s < TINY else s


def codes_ref(x, scale) -> np.ndarray:
    """int8 codes of float32 values for a given scale (zeros for scale 0 or NaN)."""
    x = np.asarray(x, dtype=F32)
    if not scale > 0:
        return np.zeros(x.shape, np.int8)
    inv = F32(1) / F32(scale)
    return np.clip(np.rint(x * inv), -127, 127).astype(np.int8)


def quantize_rows_ref(X):
    """(codes int8, scales float32) of the rows of a float32 matrix."""
    X = np.asarray(X, dtype=F32)
    scales = np.array([scale_ref(np.max(np.abs(r))) if not np.isnan(r).any() else F32(np.nan)
                       for r in X], dtype=F32)
    codes = np.stack([codes_ref(r, s) for r, s in zip(X, scales)]) if len(X) else \
        np.zeros(X.shape, np.int8)
    return codes, scales


def int8_linear_ref(X, W, w_scale, bias=None):
    """(y, magnitude of the product before the bias) in float64."""
    codes, sx = quantize_rows_ref(X)
    acc = codes.astype(np.float64) @ np.asarray(W, dtype=np.float64).T
    prod = acc * sx.astype(np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :]
    return (prod if bias is None else prod + np.asarray(bias, np.float64)), np.abs(prod)


class Kv8Ref:
    """The paged cache: codes and scales as the definition gives them."""

    def __init__(self, pages, heads, head_dim, block):
        self.block = block
        self.codes = [np.zeros((pages, heads, block, head_dim), np.int8) for _ in range(2)]
        self.scale = [np.zeros((pages, heads), F32) for _ in range(2)]

    def append(self, kv, cu, before, table):
        for which in range(2):
            x, codes, scale = np.asarray(kv[which], F32), self.codes[which], self.scale[which]
            for b in range(len(before)):
                n = cu[b + 1] - cu[b]
                pos = before[b]
                while pos < before[b] + n:
                    page, lo = table[b][pos // self.block], pos % self.block
                    hi = min(self.block, lo + before[b] + n - pos)
                    row = cu[b] + pos - before[b]
                    for h in range(codes.shape[1]):
                        new = x[row:row + hi - lo, h]
                        s = F32(np.nan) if np.isnan(new).any() else scale_ref(np.abs(new).max())
                        if lo > 0:
                            old = scale[page, h]
                            s = F32(np.nan) if np.isnan(old) or np.isnan(s) else max(s, old)
                            if s != old:
                                ratio = old / s if s > 0 else F32(0)
                                kept = codes[page, h, :lo].astype(F32) * F32(ratio)
                                codes[page, h, :lo] = (np.rint(kept) if ratio > 0 else 0)
                        codes[page, h, lo:hi] = codes_ref(new, s)
                        scale[page, h] = s
                    pos += hi - lo

    def tokens(self, which, b, start, stop, table):
        """Dequantized tokens [start, stop) of a sequence, float64 [n, heads, head_dim]."""
        at = np.arange(start, stop)
        page = np.asarray(table[b])[at // self.block] if len(at) else np.zeros(0, int)
        c = self.codes[which][page, :, at % self.block].astype(np.float64)
        return c * self.scale[which][page].astype(np.float64)[..., None]


def attention_ref(cache, q, cu, lens, table, scale, window=0):
    """(out, lse, tol_out, tol_lse) in float64: the tolerances are bounds on what
    the kernel's arithmetic may be off before the result is rounded to its type.

    Scores are sums of head_dim exact products in fp32 and two more products, so
    each is off by at most (d + 4) 2^-23 of the sum of magnitudes, B; that is an
    absolute error of a logarithm, to which the exponential adds 2^-20.
    Probabilities are rounded to fp16 (half a step, 2^-11), or, far below the
    largest, to multiples of 2^-24 / 2^7 of the largest scale that the row sees
    (half a step is 2^-32 of 127 times it, for each key)."""
    q = np.asarray(q, np.float64)
    rows, heads, d = q.shape
    kvh = cache.codes[0].shape[1]
    out, lse = np.zeros(q.shape), np.full((rows, heads), -np.inf)
    tol_o, tol_l = np.zeros(q.shape), np.full((rows, heads), 2.0 ** -20)
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        k = cache.tokens(0, b, 0, lens[b], table)
        v = cache.tokens(1, b, 0, lens[b], table)
        page = np.asarray(table[b])[np.arange(lens[b]) // cache.block]
        vs = np.asarray(cache.scale[1], np.float64)[page]          # [keys, kv heads]
        for i in range(n):
            p = lens[b] - n + i
            lo = max(0, p + 1 - window) if window else 0
            for h in range(heads):
                kk, vv = k[lo:p + 1, h // (heads // kvh)], v[lo:p + 1, h // (heads // kvh)]
                row = q[cu[b] + i, h]
                s = kk @ row * scale
                seen = vs[lo:p + 1, h // (heads // kvh)]
                vmax = 127 * seen[np.isfinite(seen)].max(initial=0.0)
                mag = (np.abs(kk) @ np.abs(row)).max() * abs(scale)
                e = np.exp(s - s.max())
                l = e.sum()
                out[cu[b] + i, h] = e @ vv / l
                lse[cu[b] + i, h] = s.max() + np.log(l)
                off = 2 * (d + 4) * 2.0 ** -23 * mag + 2.0 ** -20
                tol_o[cu[b] + i, h] = (e @ np.abs(vv) / l * (2.0 ** -11 + 2 * off)
                                       + len(e) * 2.0 ** -32 * vmax)
                tol_l[cu[b] + i, h] = off + 2.0 ** -22 * abs(lse[cu[b] + i, h])
    return out, lse, tol_o, tol_l
