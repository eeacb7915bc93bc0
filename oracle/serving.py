"""float64 CPU oracle of the serving operators (rglru_add_rmsnorm, rglru_linear_w4, rglru_paged_append,
rglru_paged_attention) -- TEST INFRASTRUCTURE, written from the formulas with plain loops.

8-bit values are e4m3 codes with power-of-two scales: x is held as c * 2^e, e the smallest exponent in
[-100, 120] with amax <= 448 * 2^e, c the nearest e4m3 value (ties to even).  e4m3: a sign, 4 exponent bits
(bias 7), 3 mantissa bits; the largest value is 448 (0x7e), 0x7f is NaN, the smallest step 2^-9.
"""
from __future__ import annotations

import numpy as np

from oracle import mqa

MIN_EXP, MAX_EXP = -100, 120


def e4m3_table() -> np.ndarray:
    """The value of each of the 256 codes."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


TABLE = e4m3_table()


def scale_of(amax) -> np.ndarray:
    """The smallest 2^e, e in [-100, 120], with amax <= 448 * 2^e."""
    amax = np.asarray(amax, np.float64)
    m, e = np.frexp(np.where(np.isfinite(amax) & (amax > 0), amax, 1.0))
    e = np.where(m <= 0.875, e - 9, e - 8)
    e = np.where(amax == 0, MIN_EXP, np.where(np.isinf(amax), MAX_EXP, e))
    return np.exp2(np.clip(e, MIN_EXP, MAX_EXP).astype(np.float64))


def amax_of(x, axis) -> np.ndarray:
    """Largest magnitude; NaN does not count."""
    a = np.abs(np.asarray(x, np.float64))
    return np.where(np.isnan(a), 0.0, a).max(axis=axis)


def round_e4m3(x) -> np.ndarray:
    """The nearest e4m3 value, ties to even, saturating at 448; NaN stays."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(np.where(np.isfinite(a) & (a > 0), a, 1.0))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.copysign(np.rint(a / step) * step, x)


def add_rmsnorm(h, weight, eps) -> np.ndarray:
    h = np.asarray(h, np.float64)
    return h / np.sqrt((h * h).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def unpack_w4(W) -> np.ndarray:
    """[N, K / 2] bytes -> [N, K] integers q - 8."""
    W = np.asarray(W)
    q = np.empty((W.shape[0], 2 * W.shape[1]), np.float64)
    q[:, 0::2] = W & 15
    q[:, 1::2] = W >> 4
    return q - 8


def linear_w4(x, W, W_scale, bias=None):
    """(out, sum_k |s q x|): the second is what a bound on the sum's rounding goes by."""
    x = np.asarray(x, np.float64)
    w = unpack_w4(W)
    w = w * np.repeat(np.asarray(W_scale, np.float64), w.shape[1] // W_scale.shape[1], axis=1)
    out = x @ w.T
    return (out if bias is None else out + np.asarray(bias, np.float64)), np.abs(x) @ np.abs(w).T


def append(qkv, cu, ctx, table, k, ks, v, vs, H, base=10000.0):
    """q [rows, H, D] rotated (rows behind the last sequence are NaN: not written) and copies of the cache
    (values, not codes: k / ks etc. are c and s) after the call; also k's and v's values before rounding, NaN where
    nothing was written."""
    qkv = np.asarray(qkv, np.float64)
    P, Hkv, ps, D = k.shape
    x = qkv.reshape(qkv.shape[0], H + 2 * Hkv, D)
    q = np.full((qkv.shape[0], H, D), np.nan)
    pools = {"k": [np.array(k, np.float64), np.array(ks, np.float64), np.full(k.shape, np.nan)],
             "v": [np.array(v, np.float64), np.array(vs, np.float64), np.full(k.shape, np.nan)]}
    for i in range(len(ctx)):
        a, b = int(cu[i]), int(cu[i + 1])
        if a == b:
            continue
        pos = ctx[i] + np.arange(b - a)
        y = mqa.rope(x[a:b, :H + Hkv], pos, base)
        q[a:b] = y[:, :H]
        for name, val in (("k", y[:, H:]), ("v", x[a:b, H + Hkv:])):
            c, s, raw = pools[name]
            for j in np.unique(pos // ps):
                page = int(table[i, j])
                if not 0 <= page < P:
                    continue
                rows = np.nonzero(pos // ps == j)[0]
                slots = pos[rows] % ps
                for h in range(Hkv):
                    new = scale_of(amax_of(val[rows, h], None))
                    if slots[0] > 0:
                        new = max(new, s[page, h])
                        if new != s[page, h]:
                            c[page, h, :slots[0]] = round_e4m3(c[page, h, :slots[0]] * (s[page, h] / new))
                    s[page, h] = new
                    c[page, h, slots] = round_e4m3(val[rows, h] / new)
                    raw[page, h, slots] = val[rows, h]
    return q, pools


def attention(q, cu, ctx, table, k, ks, v, vs, window, scale):
    """(out, bound): out [rows, H, D] (NaN rows behind the last sequence), and bound with the same shape, sum_p
    softmax_p |v_p| (the size that a relative error of the probabilities acts on), and the largest sum_d |q k| *
    scale of each (row, head): what a bound on the scores' rounding goes by.  k, v are code values, ks, vs scales."""
    q = np.asarray(q, np.float64)
    rows, H, D = q.shape
    P, Hkv, ps, _ = k.shape
    out, size, smax = np.full(q.shape, np.nan), np.zeros(q.shape), np.zeros((rows, H))
    for i in range(len(ctx)):
        for t in range(int(cu[i + 1]) - int(cu[i])):
            row, pos = int(cu[i]) + t, int(ctx[i]) + t
            p = np.arange(max(0, pos - window + 1), pos + 1)
            page = np.asarray(table)[i, p // ps].astype(np.int64)
            ok = (page >= 0) & (page < P)
            p, page = p[ok], page[ok]
            for h in range(H):
                g = h // (H // Hkv)
                if len(p) == 0:
                    out[row, h] = 0
                    continue
                kk = np.asarray(k[page, g, p % ps], np.float64) * ks[page, g][:, None]
                vv = np.asarray(v[page, g, p % ps], np.float64) * vs[page, g][:, None]
                s = kk @ q[row, h] * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                out[row, h] = w @ vv
                size[row, h] = w @ np.abs(vv)
                smax[row, h] = (np.abs(kk) @ np.abs(q[row, h])).max() * scale
    return out, size, smax
