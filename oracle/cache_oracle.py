"""Float64 reference of the operators around the paged cache: per-head norm with rotation, the
cache's formats, and the attention of drafted tokens.  Test infrastructure, written from the
definitions in include/bsa.h; it shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

BF16, E4M3, E2M1 = 0, 1, 2


# ---------------------------------------------------------------- norm and rotation

def norm_rope(x, weight, positions, inv_freq, eps, rotary, pairs, norm):
    """Rows x [tokens, heads, d] (float64) normed and rotated; also the size |a| + |b| of each
    element's pair after the norm (the element itself where it is not rotated)."""
    x = np.asarray(x, dtype=np.float64)
    y = x
    if norm:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            y = y * weight
    out, size = y.copy(), np.abs(y)
    half = rotary // 2
    if half:
        ang = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        i = 2 * np.arange(half) if pairs else np.arange(half)
        j = i + 1 if pairs else i + half
        out[..., i] = y[..., i] * c - y[..., j] * s
        out[..., j] = y[..., j] * c + y[..., i] * s
        size[..., i] = size[..., j] = np.abs(y[..., i]) + np.abs(y[..., j])
    return out, size


# ---------------------------------------------------------------- the cache's formats

def _code_values(exp_bits, frac_bits, bias, codes):
    v = np.zeros(codes)
    for c in range(codes):
        e, m = c >> frac_bits, c & ((1 << frac_bits) - 1)
        v[c] = m * 2.0 ** (1 - bias - frac_bits) if e == 0 else (1 + m / 2 ** frac_bits) * 2.0 ** (e - bias)
    return v


E4M3_VALUES = _code_values(4, 3, 7, 127)      # codes 0 .. 126 (127 is NaN); sign is bit 7
E2M1_VALUES = _code_values(2, 1, 1, 8)        # codes 0 .. 7; sign is bit 3


def _nearest(a, values):
    """Index of the value nearest to a >= 0, ties to the even code, saturated at the largest."""
    hi = np.clip(np.searchsorted(values, a), 1, len(values) - 1)
    lo = hi - 1
    dl, dh = a - values[lo], values[hi] - a
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def _least_exponent(amax, most):
    """The least k >= -126 with amax <= most * 2^k."""
    k = np.full(amax.shape, -126)
    pos = amax > 0
    g = np.zeros(amax.shape, dtype=np.int64)
    g[pos] = np.floor(np.log2(amax[pos] / most)).astype(np.int64) - 1
    for _ in range(3):                                     # the estimate is at most a few too low
        g = np.where(pos & (np.ldexp(most, g) < amax), g + 1, g)
    return np.where(pos, np.maximum(k, g), -126)


def quantise(x, fmt):
    """Rows x [..., d] as the bytes the cache holds: (codes [..., row] uint8, row exponents [...] uint8 or
    None, group scales [..., d / 16] uint8 or None)."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == BF16:
        bits = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32) >> 16
        return np.ascontiguousarray(bits.astype(np.uint16)).view(np.uint8), None, None
    bad = ~np.isfinite(x)                                  # NaN's code; in E2M1 a NaN scale for the whole group
    if fmt == E2M1:
        bad = bad.reshape(*x.shape[:-1], x.shape[-1] // 16, 16).any(-1, keepdims=True) & np.ones(16, bool)
        bad = bad.reshape(x.shape)
    x = np.where(bad, 0.0, x)
    amax = np.abs(x).max(-1)
    k = _least_exponent(amax, 448.0 if fmt == E4M3 else 2688.0)
    y = x * np.ldexp(1.0, -k)[..., None]
    sign = np.signbit(x)
    if fmt == E4M3:
        c = np.where(bad, 127, _nearest(np.abs(y), E4M3_VALUES) + 128 * sign)
        return c.astype(np.uint8), (k + 127).astype(np.uint8), None
    g = y.reshape(*y.shape[:-1], y.shape[-1] // 16, 16)
    s8 = _nearest(np.abs(g).max(-1) / 6.0, E4M3_VALUES)
    s = E4M3_VALUES[s8][..., None]
    s8 = np.where(bad.reshape(g.shape)[..., 0], 127, s8)
    c = np.where(s > 0, _nearest(np.abs(g) / np.where(s > 0, s, 1.0), E2M1_VALUES), 0)
    c = (c + 8 * (sign.reshape(g.shape) & (s > 0))).reshape(y.shape).astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), (k + 127).astype(np.uint8), s8.astype(np.uint8)


def dequantise(codes, exps, groups, fmt):
    """Float64 values of the held rows."""
    if fmt == BF16:
        u = np.ascontiguousarray(codes).view(np.uint16).astype(np.uint32) << 16
        return u.view(np.float32).astype(np.float64)
    p = np.ldexp(1.0, exps.astype(np.int64) - 127)[..., None]
    if fmt == E4M3:
        v = np.concatenate([E4M3_VALUES, [np.nan]])[codes & 127]
        return np.where(codes & 128, -v, v) * p
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = E2M1_VALUES[c & 7]
    v = np.where(c & 8, -v, v).reshape(*c.shape[:-1], c.shape[-1] // 16, 16)
    s = np.concatenate([E4M3_VALUES, [np.nan]])[groups & 127]
    return (v * s[..., None]).reshape(c.shape) * p


def held(x, fmt):
    """The values a cache of this format holds for rows x."""
    return dequantise(*quantise(x, fmt), fmt)


# ---------------------------------------------------------------- drafted tokens

def tree_attention(q, k_new, v_new, k, v, parents, scale):
    """One sequence and one KV head: q [t, g, d] drafted queries, k_new, v_new [t, d], k, v [n, d] the
    cached keys it attends to, parents [t] (-1: root).  Returns o [t, g, d], lse [t, g], and for error
    bounds sum p |v| / sum p [t, g, d] and the largest scale * sum |q_x k_x| of a visible key [t, g]."""
    t, grp, d = q.shape
    keys, vals = np.concatenate([k, k_new]), np.concatenate([v, v_new])
    n = len(k)
    o, a = np.zeros((t, grp, d)), np.zeros((t, grp, d))
    lse, reach = np.zeros((t, grp)), np.zeros((t, grp))
    for i in range(t):
        path, p = [], i
        while p >= 0:
            path.append(n + p)
            p = parents[p]
        at = np.concatenate([np.arange(n), np.array(sorted(path))])
        kk, vv = keys[at], vals[at]
        s = scale * q[i] @ kk.T
        m = s.max(-1, keepdims=True)
        e = np.exp(s - m)
        z = e.sum(-1, keepdims=True)
        o[i], a[i] = e @ vv / z, e @ np.abs(vv) / z
        lse[i] = (m + np.log(z))[:, 0]
        reach[i] = (scale * np.abs(q[i]) @ np.abs(kk).T).max(-1)
    return o, lse, a, reach
