"""fp64 definitions of the attention operators (numpy, for tests): the norm and
rotation of queries and keys, and attention with a sliding window and first
tokens that stay visible."""

from __future__ import annotations

import numpy as np


def rows_of(x, cu):
    """(batch row, first token, end) of every sequence."""
    if cu is None:
        return [(b, 0, x.shape[1]) for b in range(x.shape[0])]
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def positions_of(x, cu):
    pos = np.zeros(x.shape[:2], dtype=np.int64)
    for b, t0, t1 in rows_of(x, cu):
        pos[b, t0:t1] = np.arange(t1 - t0)
    return pos


def _pair_index(n, interleaved):
    j = np.arange(n)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + n)


def _angles(pos, inv_freq):
    # exact products of an integer and an fp32 frequency in extended precision,
    # reduced before they become fp64
    turn = np.asarray(pos, dtype=np.longdouble)[..., None] * np.asarray(inv_freq, dtype=np.longdouble)
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    return np.asarray(turn - two_pi * np.floor(turn / two_pi), dtype=np.float64)[:, :, None, :]


def _turn(x, angle, interleaved):
    y = x.copy()
    u, v = _pair_index(angle.shape[-1], interleaved)
    c, s = np.cos(angle), np.sin(angle)
    y[..., u] = x[..., u] * c - x[..., v] * s
    y[..., v] = x[..., v] * c + x[..., u] * s
    return y


def rope_fwd(x, weight, inv_freq, pos, eps=1e-6, interleaved=False):
    """One of q and k: (B, T, heads, d)."""
    w = 1.0 if weight is None else weight
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return n if inv_freq is None else _turn(n, _angles(pos, inv_freq), interleaved)


def rope_bwd(x, weight, inv_freq, pos, dy, eps=1e-6, interleaved=False):
    """Returns (dx, dweight)."""
    w = np.ones(x.shape[-1]) if weight is None else weight
    g = dy if inv_freq is None else _turn(dy, -_angles(pos, inv_freq), interleaved)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdims=True))
    return dx, (g * n).reshape(-1, x.shape[-1]).sum(0)


def _visible(n, window, sinks):
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def window_fwd(q, k, v, window, sinks=0, scale=None, cu=None):
    """(out, log-sum-exp of the scores (B, H, T))."""
    B, T, H, d = q.shape
    G = H // k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    out, lse = np.zeros(q.shape[:3] + (v.shape[-1],)), np.zeros((B, H, T))
    for b, t0, t1 in rows_of(q, cu):
        see = _visible(t1 - t0, window, sinks)
        for h in range(H):
            if t1 == t0:
                continue
            s = np.where(see, q[b, t0:t1, h] @ k[b, t0:t1, h // G].T * scale, -np.inf)
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            z = e.sum(1, keepdims=True)
            out[b, t0:t1, h] = e / z @ v[b, t0:t1, h // G]
            lse[b, h, t0:t1] = (top + np.log(z))[:, 0]
    return out, lse


def window_bwd(q, k, v, d_out, window, sinks=0, scale=None, cu=None):
    B, T, H, d = q.shape
    G = H // k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    res = {"dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    for b, t0, t1 in rows_of(q, cu):
        see = _visible(t1 - t0, window, sinks)
        for h in range(H):
            if t1 == t0:
                continue
            qq, kk, vv, g = q[b, t0:t1, h], k[b, t0:t1, h // G], v[b, t0:t1, h // G], d_out[b, t0:t1, h]
            s = np.where(see, qq @ kk.T * scale, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            dp = g @ vv.T
            ds = p * (dp - (p * dp).sum(1, keepdims=True)) * scale
            res["dq"][b, t0:t1, h] += ds @ kk
            res["dk"][b, t0:t1, h // G] += ds.T @ qq
            res["dv"][b, t0:t1, h // G] += p.T @ g
    return res


def cache_row(p, window, sinks):
    """The cache row of the token at position p."""
    return p if p < sinks else sinks + (p - sinks) % window


def window_step(q, k, v, k_cache, v_cache, lengths, sinks=0, scale=None, slots=None):
    """One token per row: (out, k_cache, v_cache), the caches as copies."""
    kc, vc = k_cache.copy(), v_cache.copy()
    B, H, d = q.shape
    R, Hk = kc.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    out = np.zeros(q.shape)
    for b in range(B):
        s = b if slots is None else slots[b]
        if s < 0:
            continue
        p = int(lengths[b])
        at = cache_row(p, R - sinks, sinks)
        kc[s, at], vc[s, at] = k[b], v[b]
        n = min(p + 1, R)
        for h in range(H):
            x = kc[s, :n, h // (H // Hk)] @ q[b, h] * scale
            e = np.exp(x - x.max())
            out[b, h] = e / e.sum() @ vc[s, :n, h // (H // Hk)]
    return out, kc, vc
