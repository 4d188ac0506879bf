"""Float64 references of the calls on heads, with error scales (numpy only): the norm and rotation of
q and k, the 8-bit cache (a model of its blocks, exact) and attention over what a cache holds.

Bounds as in :mod:`oracle.layers`: they follow the roundings of the formula term by term.
"""
from __future__ import annotations

import numpy as np

from oracle.layers import U, _cap_err

HALF = 2.0 ** -11   # unit round-off of half precision
BLOCK = 64


# ------------------------------------------------------------------ norm and rotation

def _turn(x, R, pairs, c, s):
    """x (B, L, H, D) turned by angles whose cosine and sine are c, s (B, L, R / 2); and the sum of
    magnitudes of each result."""
    y, m = x.copy(), np.abs(x)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if pairs else (slice(0, R // 2), slice(R // 2, R))
    c, s = c[:, :, None], s[:, :, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    m[..., a] = m[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, m


def angles(pos, f):
    """cos and sin of pos (B, L) times f (n): the product exact, reduced in extended precision."""
    t = pos.astype(np.longdouble)[:, :, None] * f.astype(np.longdouble)
    return np.cos(t).astype(np.float64), np.sin(t).astype(np.float64)


def qk_norm(x, w, pos, f, pairs, eps):
    """y and its bound for rows x (B, L, H, D).  rstd: a sum of D squares (at most D additions deep),
    a product, an addition, a root and a quotient; two products; cos and sin to 4 U absolute (the
    argument's and the series' roundings); three roundings of the turn."""
    D, R = x.shape[-1], 2 * len(f)
    c, s = angles(pos, f)
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y, m = _turn(x * rstd * w, R, pairs, c, s)
    return y, (0.5 * min(D, 64) + 20) * U * m


def qk_norm_bwd(dy, x, w, pos, f, pairs, eps):
    """dx, dw and their bounds."""
    D, R = x.shape[-1], 2 * len(f)
    c, s = angles(pos, f)
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * rstd
    e, m = _turn(dy, R, pairs, c, -s)
    ew, mw = e * w, m * np.abs(w)
    dx = rstd * (ew - xh * (ew * xh).mean(-1, keepdims=True))
    n = (1.5 * min(D, 64) + 40) * U
    bx = n * rstd * (mw + np.abs(xh) * (mw * np.abs(xh)).mean(-1, keepdims=True))
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    return ((dx, (e * xh).sum((0, 1, 2))),
            (bx, (n + (rows + 40) * U) * (m * np.abs(xh)).sum((0, 1, 2))))


# ------------------------------------------------------------------ the cache

def e4m3(x):
    """Nearest value of 4 exponent and 3 mantissa bits (ties to even), magnitudes up to 448."""
    a = np.minimum(np.abs(x), 448.0)
    step = 2.0 ** (np.maximum(np.frexp(a)[1] - 1, -6) - 3)
    return np.sign(x) * np.rint(a / step) * step


def rounded(x, code):
    if code == "int8":
        return np.where(np.isnan(x), 0.0, np.rint(np.clip(x, -127, 127)))
    return np.where(np.isnan(x), np.nan, e4m3(x))


def exponent(top, code):
    """The smallest in -60 .. 60 with top <= Q 2^e, elementwise."""
    q = 127.0 if code == "int8" else 448.0
    m, e = np.frexp(top / q)
    return np.clip(np.where(top > 0, e - (m == 0.5), -60), -60, 60).astype(int)


class Cache:
    """What sc_cache_write and sc_cache_read do, block by block."""

    def __init__(self, B, N, P, H, D, code, table=None):
        self.B, self.N, self.P, self.H, self.D, self.code = B, N, P, H, D, code
        self.table = np.arange(B * N).reshape(B, N) if table is None else table
        self.codes = np.zeros((2, P, BLOCK, H, D))
        self.exps = np.full((2, P, H), -60)   # a scale of 0, as memory may hold it, counts as the lowest

    def write(self, k, v, lens):
        L = k.shape[1]
        for b in range(self.B):
            end = int(lens[b])
            start = end - L
            for i in range(self.N):
                p = self.table[b, i]
                a, z = max(start, BLOCK * i, 0) - BLOCK * i, min(end, BLOCK * i + BLOCK) - BLOCK * i
                if a >= z or not 0 <= p < self.P:
                    continue
                for s, x in enumerate((k, v)):
                    new = x[b, BLOCK * i + a - start:BLOCK * i + z - start]
                    mag = np.where(np.isfinite(new), np.abs(new), 0.0).max((0, 2))
                    e = exponent(mag, self.code)
                    if a:
                        had = self.exps[s, p]
                        e = np.maximum(e, had)
                        self.codes[s, p, :a] = rounded(self.codes[s, p, :a] * 2.0 ** (had - e)[None, :, None], self.code)
                    self.codes[s, p, a:z] = rounded(new / 2.0 ** e[None, :, None], self.code)
                    self.exps[s, p] = e

    def read(self, L, lens):
        out = np.zeros((2, self.B, L, self.H, self.D))
        live = np.zeros((self.B, L), bool)
        for b in range(self.B):
            for t in range(L):
                j = int(lens[b]) - L + t
                if not 0 <= j < BLOCK * self.N:
                    continue
                p = self.table[b, j // BLOCK]
                if 0 <= p < self.P:
                    live[b, t] = True
                    out[:, b, t] = self.codes[:, p, j % BLOCK] * 2.0 ** self.exps[:, p][..., None]
        return out[0], out[1], live


# ------------------------------------------------------------------ attention over it

def cached_attention(q, k, v, lens, scale, window=0, sinks=0, cap=0.0, slopes=None, live=None, bf16=False):
    """o, lse and their bounds; k, v (B, Lk, Hkv, D) by position, live (B, Lk): keys of no bad block."""
    B, Lq, H, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    lse, bl = np.full((B, H, Lq), -np.inf), np.zeros((B, H, Lq))
    part = 0.0 if bf16 else 2.0 ** -22   # a query value, a weight as two halves
    j = np.arange(Lk)[None]
    for b in range(B):
        p = int(lens[b]) - Lq + np.arange(Lq)[:, None]
        see = (j <= p) & (p >= 0) & (p < Lk)
        if window:
            see &= (j > p - window) | (j < sinks)
        if live is not None:
            see &= live[b][None]
        rows, cols = see.any(1), see.any(0)
        if not rows.any():
            continue
        for h in range(H):
            g = h // (H // Hkv)
            qq = np.where(rows[:, None], q[b, :, h], 0.0)
            kk, vv = (np.where(cols[:, None], x[b, :, g], 0.0) for x in (k, v))
            x = scale * (qq @ kk.T)
            mag = scale * (np.abs(qq) @ np.abs(kk).T)
            # a query value below 2^-24 halves of its row's largest is off by 2^-40 of that
            low = scale * 2.0 ** -39 * np.abs(qq).max(1, keepdims=True) * np.abs(kk).sum(1)[None]
            err = ((2 if not bf16 else 1) * D + 8) * U * mag + part * mag + low
            s = x
            if cap:
                s = cap * np.tanh(x / cap)
                err = err + _cap_err(s, cap, False)
            bias = 0.0 if slopes is None else float(slopes[h])
            s = s - bias * (p - j)
            # the exponent of a weight: its base, the block's scale (60 at most) and the bias are added
            # in turn; a base that rises leaves the roundings of what it rose by, at most twice the
            # largest score
            far = np.abs(bias * (p - j))
            top = np.where(see, np.abs(s), 0.0).max(1, keepdims=True)
            err = np.where(see, err + 8 * U * (np.abs(s) + far + top + 70), 0.0)
            s = np.where(see, s, -np.inf)
            m = np.where(rows, s.max(1, initial=-np.inf), 0.0)
            e = np.exp(s - m[:, None])
            l = np.where(rows, e.sum(1), 1.0)
            w = e / l[:, None]
            o[b, :, h] = w @ vv
            worst, n = err.max(1, initial=0.0), see.sum(1)
            rel = 2 * worst + (n + 60) * U + (HALF if bf16 else 2.0 ** -22)
            # weights under 2^-14 of half precision's range: 2^-25 / 2^7 of the row's largest contribution,
            # whose codes reach 448 times theirs
            tiny = n[:, None] * 2.0 ** -32 * 448 * (w @ np.abs(vv)).max(1, keepdims=True)
            bo[b, :, h] = rel[:, None] * (w @ np.abs(vv)) + tiny
            lse[b, h, rows] = (m + np.log(l))[rows]
            bl[b, h, rows] = (worst + (n + 16) * U + 4 * U * np.abs(np.where(rows, lse[b, h], 0.0)))[rows]
    return (o, lse), (bo, bl)
