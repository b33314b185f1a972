"""fp64 definitions of the mixer operators and their hand-derived reverse
modes (numpy, token by token; test infrastructure only).

A batch is a list of sequences: bounds() gives (batch row, start, end) of each
for dense (B, T, ...) or packed (1, T, ...) arrays.
"""

from __future__ import annotations

import numpy as np


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def act(x, kind):
    return x if kind in (None, "none") else x * sigmoid(x) if kind == "silu" else sigmoid(x)


def dact(x, kind):
    s = sigmoid(x)
    return np.ones_like(x) if kind in (None, "none") else s * (1 + x * (1 - s)) if kind == "silu" else s * (1 - s)


def bounds(B, T, cu=None):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]


# ---------------------------------------------------------------- convolution

def conv_fwd(x, w, bias=None, kind="silu", state=None, cu=None):
    B, T, D = x.shape
    W = w.shape[1]
    y = np.zeros_like(x)
    seqs = bounds(B, T, cu)
    fs = np.zeros((len(seqs), W - 1, D))
    for n, (b, t0, t1) in enumerate(seqs):
        head = np.zeros((W - 1, D)) if state is None else state[n]
        ext = np.concatenate([head, x[b, t0:t1]])
        for t in range(t1 - t0):
            p = (ext[t:t + W] * w.T).sum(0) + (0 if bias is None else bias)
            y[b, t0 + t] = act(p, kind)
        fs[n] = ext[ext.shape[0] - (W - 1):]
    return y, fs


def conv_bwd(x, w, dy, bias=None, kind="silu", state=None, cu=None, dfs=None):
    B, T, D = x.shape
    W = w.shape[1]
    seqs = bounds(B, T, cu)
    r = dict(dx=np.zeros_like(x), dweight=np.zeros_like(w), dbias=np.zeros(D),
             d_initial_state=np.zeros((len(seqs), W - 1, D)))
    for n, (b, t0, t1) in enumerate(seqs):
        head = np.zeros((W - 1, D)) if state is None else state[n]
        ext = np.concatenate([head, x[b, t0:t1]])
        dext = np.zeros_like(ext)
        if dfs is not None:
            dext[ext.shape[0] - (W - 1):] += dfs[n]
        for t in range(t1 - t0):
            p = (ext[t:t + W] * w.T).sum(0) + (0 if bias is None else bias)
            dp = dy[b, t0 + t] * dact(p, kind)
            dext[t:t + W] += dp * w.T
            r["dweight"] += (dp * ext[t:t + W]).T
            r["dbias"] += dp
        r["d_initial_state"][n] = dext[:W - 1]
        r["dx"][b, t0:t1] = dext[W - 1:]
    return r


# ----------------------------------------------------------------------- scan

def _step(dt, bias, soft):
    raw = dt if bias is None else dt + bias
    return raw, (np.logaddexp(0.0, raw) if soft else raw)


def scan_fwd(u, dt, A, B, C, D=None, z=None, dt_bias=None, soft=True, state=None, cu=None, keep=None):
    nb, T, d = u.shape
    G, N = B.shape[2:]
    _, step = _step(dt, dt_bias, soft)
    seqs = bounds(nb, T, cu)
    y = np.zeros_like(u)
    fs = np.zeros((len(seqs), d, N))
    wide = lambda v: np.repeat(v, d // G, axis=0)  # noqa: E731
    for n, (b, t0, t1) in enumerate(seqs):
        h = np.zeros((d, N)) if state is None else state[n].copy()
        for t in range(t0, t1):
            if keep is not None:
                keep[(n, t)] = h
            h = np.exp(step[b, t][:, None] * A) * h + (step[b, t] * u[b, t])[:, None] * wide(B[b, t])
            y[b, t] = (h * wide(C[b, t])).sum(1)
        fs[n] = h
    if D is not None:
        y = y + D * u
    return (y if z is None else y * act(z, "silu")), fs


def scan_bwd(u, dt, A, B, C, dout, D=None, z=None, dt_bias=None, soft=True, state=None, cu=None, dfs=None):
    nb, T, d = u.shape
    G, N = B.shape[2:]
    raw, step = _step(dt, dt_bias, soft)
    seqs = bounds(nb, T, cu)
    keep = {}
    y, _ = scan_fwd(u, dt, A, B, C, D, None, dt_bias, soft, state, cu, keep)
    dy = dout if z is None else dout * act(z, "silu")
    r = dict(du=np.zeros_like(u), ddt=np.zeros_like(u), dA=np.zeros_like(A), dB=np.zeros_like(B),
             dC=np.zeros_like(C), d_initial_state=np.zeros((len(seqs), d, N)))
    r["dz"] = None if z is None else dout * y * dact(z, "silu")
    wide = lambda v: np.repeat(v, d // G, axis=0)  # noqa: E731
    part = lambda v: v.reshape(G, d // G, N).sum(1)  # noqa: E731
    for n, (b, t0, t1) in enumerate(seqs):
        g = np.zeros((d, N)) if dfs is None else dfs[n].copy()
        for t in range(t1 - 1, t0 - 1, -1):
            s, x = step[b, t], step[b, t] * u[b, t]
            a = np.exp(s[:, None] * A)
            h = a * keep[(n, t)] + x[:, None] * wide(B[b, t])
            e = g + dy[b, t][:, None] * wide(C[b, t])
            r["dC"][b, t] = part(dy[b, t][:, None] * h)
            r["dB"][b, t] = part(e * x[:, None])
            dx = (e * wide(B[b, t])).sum(1)
            g = a * e
            q = g * keep[(n, t)]
            r["dA"] += q * s[:, None]
            r["ddt"][b, t] = (q * A).sum(1) + dx * u[b, t]
            r["du"][b, t] = dx * s
        r["d_initial_state"][n] = g
    if D is not None:
        r["du"] += D * dy
    if soft:
        r["ddt"] = r["ddt"] * sigmoid(raw)
    r["dD"] = (dy * u).sum((0, 1))
    r["ddt_bias"] = r["ddt"].sum((0, 1))
    return r


# ----------------------------------------------------------------------- norm

def norm_fwd(x, w=None, b=None, gate=None, groups=1, eps=1e-6, kind="silu", center=False, gate_first=False):
    return _norm(x, w, b, gate, groups, eps, kind, center, gate_first)[0]


def _norm(x, w, b, gate, groups, eps, kind, center, gate_first):
    rows, C = x.shape
    first = gate is not None and gate_first
    xp = (x * act(gate, kind) if first else x).reshape(rows, groups, C // groups)
    xc = xp - xp.mean(-1, keepdims=True) if center else xp
    r = 1.0 / np.sqrt((xc * xc).mean(-1, keepdims=True) + eps)
    n = (xc * r).reshape(rows, C)
    v = n * (1.0 if w is None else w) + (0.0 if b is None else b)
    y = act(v, kind) if gate is None else v if first else v * act(gate, kind)
    return y, n, v, r


def norm_bwd(x, dy, w=None, b=None, gate=None, groups=1, eps=1e-6, kind="silu", center=False, gate_first=False):
    rows, C = x.shape
    first = gate is not None and gate_first
    _, n, v, r = _norm(x, w, b, gate, groups, eps, kind, center, gate_first)
    res = {}
    dv = dy * dact(v, kind) if gate is None else dy if first else dy * act(gate, kind)
    if gate is not None and not first:
        res["dgate"] = dy * v * dact(gate, kind)
    res["dweight"], res["dbias"] = (dv * n).sum(0), dv.sum(0)
    dn = (dv * (1.0 if w is None else w)).reshape(rows, groups, C // groups)
    n3 = n.reshape(dn.shape)
    d = dn - n3 * (dn * n3).mean(-1, keepdims=True)
    if center:
        d = d - dn.mean(-1, keepdims=True)
    d = (r * d).reshape(rows, C)
    if first:
        res["dgate"] = d * x * dact(gate, kind)
        d = d * act(gate, kind)
    res["dx"] = d
    return res


# ----------------------------------------------------------------------------
# gated linear recurrence
# ----------------------------------------------------------------------------

def _gated_rows(x, cu):
    if cu is None:
        return [(b, 0, x.shape[1]) for b in range(x.shape[0])]
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def _sig(x):
    return np.exp(-np.logaddexp(0.0, -x))


def gated_fwd(x, r, i, lam, rate=8.0, h0=None, cu=None):
    """h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t, token by token, with
    a_t = exp(-rate softplus(lam) sigmoid(r_t)).  Returns (h, final states)."""
    rows = _gated_rows(x, cu)
    y = np.zeros(x.shape)
    fs = np.zeros((len(rows), x.shape[2])) if h0 is None else h0.astype(np.float64).copy()
    L = -rate * np.logaddexp(0.0, lam) * _sig(r)
    a, m = np.exp(L), np.sqrt(-np.expm1(2 * L))
    for n, (b, t0, t1) in enumerate(rows):
        h = fs[n]
        for t in range(t0, t1):
            h = a[b, t] * h + m[b, t] * _sig(i[b, t]) * x[b, t]
            y[b, t] = h
        fs[n] = h
    return y, fs


def gated_bwd(x, r, i, lam, dy, rate=8.0, h0=None, cu=None, dfs=None):
    """Its reverse mode, token by token."""
    y, _ = gated_fwd(x, r, i, lam, rate, h0, cu)
    sr, si, sp = _sig(r), _sig(i), np.logaddexp(0.0, lam)
    L = -rate * sp * sr
    a, m = np.exp(L), np.sqrt(-np.expm1(2 * L))
    rows = _gated_rows(x, cu)
    res = {k: np.zeros(x.shape) for k in ("dx", "dr", "di")}
    res["dlam"] = np.zeros(lam.shape)
    d0 = np.zeros((len(rows), x.shape[2]))
    for n, (b, t0, t1) in enumerate(rows):
        c = np.zeros(x.shape[2]) if dfs is None else dfs[n].astype(np.float64)
        for t in range(t1 - 1, t0 - 1, -1):
            dh = dy[b, t] + c
            past = y[b, t - 1] if t > t0 else (np.zeros(x.shape[2]) if h0 is None else h0[n])
            at, mt = a[b, t], m[b, t]
            with np.errstate(divide="ignore", invalid="ignore"):
                slope = np.where(mt > 0, -at * at / mt, 0.0)
            dL = dh * (at * past + slope * si[b, t] * x[b, t])
            res["dx"][b, t] = dh * mt * si[b, t]
            res["di"][b, t] = dh * mt * x[b, t] * si[b, t] * (1 - si[b, t])
            res["dr"][b, t] = dL * L[b, t] * (1 - sr[b, t])
            res["dlam"] += dL * -rate * sr[b, t] * _sig(lam)
            c = at * dh
        d0[n] = c
    if h0 is not None:
        res["d_initial_state"] = d0
    return res
