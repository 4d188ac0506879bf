"""Float64 references of the layers beside the convolution, with error scales (numpy only).

Each function takes stored values widened to float64 and returns the definition's result in 64
bits and, for the tests' tolerances, how much an evaluation in float32 may differ from it: U is
the float32 unit round-off, and every bound follows the roundings of the formula term by term
(sums over n terms in any order: n U times the sum of magnitudes, less for trees).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
UB = 2.0 ** -8      # bfloat16 unit round-off (8 significant bits)
TINY = 2.0 ** -126  # smallest normal float32: what lies below may come out as 0


# ------------------------------------------------------------------ layer norm

def layernorm(x, w, b, eps):
    """y, mean, rstd and the bounds of y, mean, rstd for rows x (R, C)."""
    R, C = x.shape
    mean = x.sum(1) / C
    d = x - mean[:, None]
    var = (d * d).sum(1) / C
    rstd = 1 / np.sqrt(var + eps)
    xh = d * rstd[:, None]
    y = xh * w + b
    # every sum is at most 100 additions deep; the mean's error moves every value of the row
    top = np.abs(x).max(1, initial=0.0)
    bm = 100 * U * top
    # the sum about the moved mean: its own roundings, and bm^2 / var
    br = rstd * (120 * U + 2 * U * (top * rstd) + 4 * (bm * rstd) ** 2)
    by = 2 * (np.abs(w) * (rstd * (bm + 2 * U * top) + 4 * U)[:, None]
              + np.abs(xh * w) * (br / rstd + 8 * U)[:, None]) + 4 * U * (np.abs(b) + np.abs(y))
    return (y, mean, rstd), (by, bm, br)


def layernorm_bwd(dy, x, w, mean, rstd):
    """dx, dw, db for given statistics, and their bounds."""
    R, C = x.shape
    r = rstd[:, None]
    xh = (x - mean[:, None]) * r
    e = dy * w
    me, mx = e.mean(1, keepdims=True), (e * xh).mean(1, keepdims=True)
    dx = r * (e - me - xh * mx)
    X = (np.abs(x) + np.abs(mean)[:, None]) * r          # |xh| before cancellation
    ae, ax = np.abs(e).mean(1, keepdims=True), (np.abs(e) * X).mean(1, keepdims=True)
    bdx = 120 * U * r * (np.abs(e) + ae + X * ax)
    dw, db = (dy * xh).sum(0), dy.sum(0)
    n = (R + 100) * U
    return (dx, dw, db), (bdx, n * (np.abs(dy) * X).sum(0), n * np.abs(dy).sum(0))


# ------------------------------------------------------------------ gated recurrence

def _gates(z):
    e = np.exp(-np.abs(z))
    big, small = 1 / (1 + e), e / (1 + e)
    return np.where(z >= 0, big, small), np.where(z >= 0, small, big)


def _gate_err(z):
    """Relative error of a gate: the exponent's rounding moves exp(-|z|) by |z| U."""
    return (8 + 2 * np.minimum(np.abs(z), 104.0)) * U


def recurrence(z, u, h0):
    """h (B, L, C), hT (B, C) and the bound of both."""
    B, L, C = z.shape
    f, k = _gates(z)
    g = _gate_err(z)
    h, bound = np.zeros_like(z), np.zeros_like(z)
    s = h0.copy()
    mag, err = np.abs(h0), np.zeros_like(h0)
    for t in range(L):
        s = f[:, t] * s + k[:, t] * u[:, t]
        # a step's gates and roundings act on magnitudes; the scan adds one rounding a level
        new = f[:, t] * mag + k[:, t] * np.abs(u[:, t])
        err = f[:, t] * err + (g[:, t] + 4 * U) * new + TINY * (mag + np.abs(u[:, t]))
        mag = new
        h[:, t], bound[:, t] = s, err + 64 * U * mag
    last = bound[:, -1] if L else np.zeros_like(h0)
    return (h, s), (bound, last)


def recurrence_bwd(dh, z, u, h, h0, dhT):
    """dz, du, dh0 and their bounds."""
    B, L, C = z.shape
    f, k = _gates(z)
    ge = _gate_err(z)
    dz, du = np.zeros_like(z), np.zeros_like(z)
    bz, bu = np.zeros_like(z), np.zeros_like(z)
    c, mag, err = dhT.copy(), np.abs(dhT), np.zeros_like(dhT)
    for t in reversed(range(L)):
        prev = h[:, t - 1] if t else h0
        g = dh[:, t] + c
        gm = np.abs(dh[:, t]) + mag
        be = err + 64 * U * gm
        du[:, t], bu[:, t] = k[:, t] * g, k[:, t] * (be + (ge[:, t] + 4 * U) * np.abs(g)) + 2 * TINY * gm
        w = f[:, t] * k[:, t]
        dz[:, t] = g * (prev - u[:, t]) * w
        bz[:, t] = w * (be * np.abs(prev - u[:, t])
                        + gm * (np.abs(prev) + np.abs(u[:, t])) * (2 * ge[:, t] + 8 * U)) \
            + 2 * TINY * gm * (1 + np.abs(prev) + np.abs(u[:, t]))
        c = f[:, t] * g
        mag, err = f[:, t] * gm, f[:, t] * (err + (ge[:, t] + 4 * U) * gm) + TINY * gm
    return (dz, du, c), (bz, bu, err + 64 * U * mag)


# ------------------------------------------------------------------ attention

def visible(Lq, Lk, window, n, doc):
    """(Lq, Lk) truth values for one batch row of n keys; doc (Lk) or None."""
    p = n - Lq + np.arange(Lq)[:, None]
    j = np.arange(Lk)[None]
    see = (j <= p) & (p >= 0) & (p < n)
    if window:
        see &= j >= p - window + 1
    if doc is not None:
        own = doc[np.clip(p, 0, max(Lk - 1, 0))] if Lk else np.zeros_like(p)
        see &= (j >= own) & (doc[None] <= j)
    return see, p - j


def _cap_err(s, cap, plain):
    """Error of s = cap tanh(x / cap) beside the argument's.  From t = 1 - 2 r, r = 1 / (1 + e^2y):
    e is off by (4 y + 2) U (its argument's two roundings; an ulp), r by that times e / (1 + e) and 3
    more: 4 U of t at most, which is what a plain evaluation has.  A series near 0 makes it relative: 2 r
    / t is 1.4 at y = 0.45, where the last of them gives way: 9 U.  The products with cap and cap's
    conversion add 3 U."""
    if plain:
        return 4 * U * cap + 3 * U * np.abs(s)
    return 12 * U * np.abs(s)


def _scores(q, k, see, far, scale, cap, slope, plain=False):
    x = scale * (q @ k.T)
    mag = scale * (np.abs(q) @ np.abs(k).T)
    t = None
    s = x
    err = (q.shape[1] + 6) * U * mag
    if cap:
        t = np.tanh(x / cap)
        s = cap * t
        err = err + _cap_err(s, cap, plain)   # tanh passes on no more than its argument's error
    s = s - slope * far
    err = err + 8 * U * (np.abs(s) + np.abs(slope * far)) + 4 * U
    return np.where(see, s, -np.inf), t, np.where(see, err, 0.0)


def _each(q, k, v, Lk, H, Hkv, window, kv_len, doc):
    for b in range(q.shape[0]):
        n = Lk if kv_len is None else min(max(int(kv_len[b]), 0), Lk)
        see, far = visible(q.shape[1], Lk, window, n, None if doc is None else doc[b].astype(np.int64))
        for h in range(H):
            g = h // (H // Hkv)
            # what no row sees may hold anything: it takes no part
            rows, cols = see.any(1), see.any(0)
            yield (b, h, g, see, far, np.where(rows[:, None], q[b, :, h], 0.0),
                   np.where(cols[:, None], k[b, :, g], 0.0), np.where(cols[:, None], v[b, :, g], 0.0), rows)


def attention(q, k, v, scale, window=0, cap=0.0, slopes=None, kv_len=None, doc=None, bf16=False):
    """o (B, Lq, H, D), lse (B, H, Lq) and their bounds; bf16: weights rounded to bfloat16."""
    B, Lq, H, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    o, bo = np.zeros(q.shape), np.zeros(q.shape)
    lse, bl = np.full((B, H, Lq), -np.inf), np.zeros((B, H, Lq))
    for b, h, g, see, far, qq, kk, vv, rows in _each(q, k, v, Lk, H, Hkv, window, kv_len, doc):
        s, _, err = _scores(qq, kk, see, far, scale, cap, 0.0 if slopes is None else float(slopes[h]))
        m = np.where(rows, s.max(1, initial=-np.inf), 0.0)
        e = np.exp(s - m[:, None])
        l = e.sum(1)
        p = e / np.where(rows, l, 1.0)[:, None]
        o[b, :, h] = p @ vv
        top = err.max(1, initial=0.0)
        n = see.sum(1)
        rel = (2 * top + (n + 40) * U + (UB if bf16 else 0.0))[:, None]
        bo[b, :, h] = rel * (p @ np.abs(vv))
        lse[b, h, rows] = (m + np.log(np.where(rows, l, 1.0)))[rows]
        bl[b, h, rows] = (top + (n + 8) * U + 4 * U * np.abs(np.where(rows, lse[b, h], 0.0)))[rows]
    return (o, lse), (bo, bl)


def attention_bwd(do, q, k, v, o, lse, scale, window=0, cap=0.0, slopes=None, kv_len=None, doc=None,
                  bf16=False):
    """dq, dk, dv for given o and lse, and their bounds; bf16: P and dS rounded to bfloat16."""
    B, Lq, H, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    out = [np.zeros(t.shape) for t in (q, k, v)]
    bd = [np.zeros(t.shape) for t in (q, k, v)]
    r = UB if bf16 else 0.0
    for b, h, g, see, far, qq, kk, vv, rows in _each(q, k, v, Lk, H, Hkv, window, kv_len, doc):
        s, t, err = _scores(qq, kk, see, far, scale, cap, 0.0 if slopes is None else float(slopes[h]),
                            plain=bf16 and cap <= 64)
        dd, oo = (np.where(rows[:, None], x[b, :, h], 0.0) for x in (do, o))
        L = np.where(rows, lse[b, h], 0.0)
        p = np.exp(s - L[:, None])
        err = err + 4 * U * (1 + np.abs(L))[:, None]
        dp, delta = dd @ vv.T, (dd * oo).sum(1, keepdims=True)
        ds = p * (dp - delta)
        es = p * (err * np.abs(dp - delta)
                  + (D + 8) * U * (np.abs(dd) @ np.abs(vv).T + (np.abs(dd) * np.abs(oo)).sum(1, keepdims=True)))
        if t is not None:
            # the factor 1 - t^2 from a tanh off by 4 U, and by its argument's error over cap
            es = es * (1 - t * t) + np.abs(ds) * (16 * U + 2 * err / cap)
            ds = ds * (1 - t * t)
        es = es + r * np.abs(ds)
        ep = p * (err + r)
        n = (max(Lq, Lk) * (H // Hkv) + 40) * U
        out[0][b, :, h] = scale * (ds @ kk)
        bd[0][b, :, h] = scale * ((es + n * np.abs(ds)) @ np.abs(kk))
        out[1][b, :, g] += scale * (ds.T @ qq)
        bd[1][b, :, g] += scale * ((es + n * np.abs(ds)).T @ np.abs(qq))
        out[2][b, :, g] += p.T @ dd
        bd[2][b, :, g] += (ep + n * p).T @ np.abs(dd)
    return tuple(out), tuple(bd)
