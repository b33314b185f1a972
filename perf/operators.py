"""The sequence-mixer operators: short causal convolution, selective state
space scan, gated group norm.  For each a range of sizes, a plain form in
elementary torch operations (fp32 throughout, rounded once at the end), the
calls a user makes of this package, and the definition in fp64.

All activations are channels last, (B, T, C).  A packed batch is (1, T, C)
with int32 offsets cu_seqlens.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}
CONV_W = 4


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one decoded token for 64 sequences, q, k and v of 16 heads x 128 side by side
        {"name": "conv_step", "op": "conv_step", "B": 64, "D": 6144, "dtype": "bf16"},
        # prompts of the package's training shape, q, k and v together
        {"name": "conv_prompt", "op": "conv_fwd", "B": 4, "T": 4096, "D": 6144, "nseq": 0, "dtype": "bf16"},
        # a few ragged sequences in one packed row, an odd channel count, continued from a state
        {"name": "conv_packed_f32", "op": "conv_fwd", "B": 1, "T": 1537, "D": 1003, "nseq": 7, "dtype": "f32"},
        # gradients of the convolution over packed training documents
        {"name": "conv_backward", "op": "conv_bwd", "B": 1, "T": 16384, "D": 2048, "nseq": 12, "dtype": "bf16"},
        # one decoded token for 256 sequences
        {"name": "scan_step", "op": "scan_step", "B": 256, "D": 2048, "G": 1, "N": 16, "dtype": "bf16"},
        # prompts of the package's training shape
        {"name": "scan_prompt", "op": "scan_fwd", "B": 4, "T": 4096, "D": 2048, "G": 1, "N": 16, "nseq": 0,
         "dtype": "bf16"},
        # one long document alone: few channels, a long serial axis
        {"name": "scan_long", "op": "scan_fwd", "B": 1, "T": 65536, "D": 1024, "G": 1, "N": 16, "nseq": 0,
         "dtype": "bf16"},
        # ragged packed sequences in fp32, two groups of B and C, a wider state, an odd width per group
        {"name": "scan_packed_f32", "op": "scan_fwd", "B": 1, "T": 2501, "D": 522, "G": 2, "N": 32, "nseq": 9,
         "dtype": "f32"},
        # a training step: forward, then every gradient
        {"name": "scan_train", "op": "scan_train", "B": 2, "T": 4096, "D": 2048, "G": 1, "N": 16, "nseq": 0,
         "dtype": "bf16"},
        # the output norm of one decoded token, 64 sequences x 16 heads
        {"name": "norm_decode", "op": "norm_fwd", "rows": 64, "C": 2048, "groups": 16, "gated": True,
         "gate_first": False, "center": False, "dtype": "bf16"},
        # the output norm over prompts
        {"name": "norm_prompt", "op": "norm_fwd", "rows": 16384, "C": 2048, "groups": 16, "gated": True,
         "gate_first": False, "center": False, "dtype": "bf16"},
        # its gradients, gate before the norm and one group over all channels
        {"name": "norm_backward", "op": "norm_bwd", "rows": 16384, "C": 2048, "groups": 1, "gated": True,
         "gate_first": True, "center": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A channel count: often a multiple of 64, else anything."""
    d = _log(rng, lo, hi)
    if rng.random() < 0.6:
        d = max(64, d // 64 * 64)
    return d + 1 if d == 3072 else d


def draw(rng):
    op = rng.choice(["conv_step", "conv_fwd", "conv_bwd", "scan_step", "scan_fwd", "scan_fwd", "scan_train",
                     "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv_step":
        return {"op": op, "B": _log(rng, 1, 1024), "D": _width(rng, 64, 8192), "dtype": dtype}
    if op == "scan_step":
        N = rng.choice([8, 16, 32, 64, 128])
        return {"op": op, "B": _log(rng, 1, max(2, 4096 // N)), "D": _width(rng, 64, 4096), "G": 1, "N": N,
                "dtype": dtype}
    if op in ("norm_fwd", "norm_bwd"):
        groups = rng.choice([1, 1, 2, 8, 16])
        size = _log(rng, 32, 8192 // groups)
        if rng.random() < 0.6:
            size = max(32, size // 32 * 32)
        if size * groups == 3072:
            size += 1
        rows = _log(rng, 1, min(32768, (1 << (25 if dtype == "bf16" else 24)) // (size * groups)))
        gated = rng.random() < 0.75
        return {"op": op, "rows": rows, "C": size * groups, "groups": groups, "gated": gated,
                "gate_first": gated and rng.random() < 0.4, "center": rng.random() < 0.3, "dtype": dtype}
    if op in ("conv_fwd", "conv_bwd"):
        D = _width(rng, 64, 8192)
        tokens = _log(rng, 1, min(65536, (1 << 25) // D))
        G, N = 0, 0
    else:
        G, N = rng.choice([(1, 8), (1, 16), (1, 16), (1, 16), (1, 32), (2, 16), (1, 64), (1, 128)])
        D = _width(rng, 64 * G, 4096) // G * G
        most = ((1 << 25) if op == "scan_fwd" else (1 << 24)) * 16 // max(N, 16) // D
        tokens = _log(rng, 1, max(1, min(65536, most)))
    case = {"op": op, "D": D, "dtype": dtype}
    if N:
        case.update(G=G, N=N)
    if rng.random() < 0.4 and tokens > 8:
        case.update(B=1, T=tokens, nseq=_log(rng, 1, min(64, tokens // 4)))
    else:
        B = _log(rng, 1, min(16, tokens))
        case.update(B=B, T=tokens // B, nseq=0)
    return case


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _offsets(seed, T, nseq):
    """Offsets of nseq ragged sequences (some may hold one token or none)."""
    rng = random.Random(seed)
    return [0] + sorted(rng.randint(0, T) for _ in range(nseq - 1)) + [T]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dtype = DTYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * scale).to(to)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32) * (hi - lo) + lo

    s = dict(case)
    if op.startswith("norm"):
        rows, C = case["rows"], case["C"]
        # x is the mixer's output; the gate is one half of the input projection, a strided view
        s["x"] = normal(rows, C, scale=0.7)
        s["gate"] = normal(rows, 2 * C)[:, C:] if case["gated"] else None
        s["weight"] = uniform(0.5, 1.5, C)
        s["bias"] = uniform(-0.2, 0.2, C) if case["center"] else None
        if op == "norm_bwd":
            s["d_out"] = normal(rows, C)
        return s
    D = case["D"]
    if op.startswith("conv"):
        s["weight"] = uniform(-0.5, 0.5, D, CONV_W)
        s["bias"] = uniform(-0.1, 0.1, D)
        if op == "conv_step":
            s["x"] = normal(case["B"], D)
            s["state"] = normal(case["B"], CONV_W - 1, D)
            s["out_state"] = torch.empty_like(s["state"])
            return s
        s["x"] = normal(case["B"], case["T"], D)
        s["cu"] = None
        s["h0"] = None
        if case["nseq"]:
            s["cu"] = torch.tensor(_offsets(seed, case["T"], case["nseq"]), dtype=torch.int32, device=dev)
            s["h0"] = normal(case["nseq"], CONV_W - 1, D)
        if op == "conv_bwd":
            s["d_out"] = normal(case["B"], case["T"], D)
        return s
    G, N = case["G"], case["N"]
    # A = -(1 .. N) with some spread per channel; step sizes of 0.001 to 0.1, as trained models start from
    s["A"] = -torch.arange(1, N + 1, device=dev, dtype=torch.float32) * uniform(0.6, 1.4, D, N)
    s["Dskip"] = uniform(0.5, 1.5, D)
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), D))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    rank = (D + 15) // 16
    if op == "scan_step":
        B = case["B"]
        s["u"] = normal(B, D, scale=0.6)
        s["dt"] = normal(B, D)
        s["z"] = normal(B, 2 * D)[:, D:]
        proj = normal(B, rank + 2 * G * N)
        s["Bm"] = proj[:, rank:rank + G * N].unflatten(1, (G, N))
        s["Cm"] = proj[:, rank + G * N:].unflatten(1, (G, N))
        s["state"] = normal(B, D, N, scale=0.3, to=torch.float32)
        s["out_state"] = torch.empty_like(s["state"])
        return s
    B, T = case["B"], case["T"]
    s["u"] = normal(B, T, D, scale=0.6)
    s["dt"] = normal(B, T, D)
    s["z"] = normal(B, T, 2 * D)[..., D:]             # half of the input projection
    proj = normal(B, T, rank + 2 * G * N)             # step rank, B and C side by side
    s["Bm"] = proj[..., rank:rank + G * N].unflatten(2, (G, N))
    s["Cm"] = proj[..., rank + G * N:].unflatten(2, (G, N))
    s["cu"] = None
    s["h0"] = None
    if case["nseq"]:
        s["cu"] = torch.tensor(_offsets(seed, T, case["nseq"]), dtype=torch.int32, device=dev)
        s["h0"] = normal(case["nseq"], D, N, scale=0.3, to=torch.float32)
    if op == "scan_train":
        s["d_out"] = normal(B, T, D)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        from linear_attention_sequence_chunked_gb300 import mixer
        if op == "conv_step":
            y = mixer.short_conv_step(s["x"], s["state"], s["weight"], s["bias"], out_state=s["out_state"])
            return {"y": y, "state": s["out_state"]}
        if op == "conv_fwd":
            y, fs = mixer.short_conv_fwd(s["x"], s["weight"], s["bias"], initial_state=s["h0"], cu_seqlens=s["cu"],
                                         output_final_state=True)
            return {"y": y, "state": fs}
        if op == "conv_bwd":
            return mixer.short_conv_bwd(s["x"], s["weight"], s["d_out"], s["bias"], initial_state=s["h0"],
                                        cu_seqlens=s["cu"])
        if op == "scan_step":
            y = mixer.ssm_scan_step(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], D=s["Dskip"], z=s["z"],
                                    dt_bias=s["dt_bias"], out_state=s["out_state"])
            return {"y": y, "state": s["out_state"]}
        if op == "scan_fwd":
            y, fs = mixer.ssm_scan_fwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["Dskip"], z=s["z"],
                                       dt_bias=s["dt_bias"], initial_state=s["h0"], cu_seqlens=s["cu"])
            return {"y": y, "state": fs}
        if op == "scan_train":
            kw = dict(D=s["Dskip"], z=s["z"], dt_bias=s["dt_bias"], initial_state=s["h0"], cu_seqlens=s["cu"])
            y, fs, saved = mixer.ssm_scan_fwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], save_for_backward=True, **kw)
            g = mixer.ssm_scan_bwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["d_out"], saved=saved, **kw)
            return {"y": y, "state": fs, **g}
        kw = dict(bias=s["bias"], gate=s["gate"], groups=s["groups"], center=s["center"], gate_first=s["gate_first"])
        if op == "norm_fwd":
            return mixer.group_norm_fwd(s["x"], s["weight"], **kw)
        return mixer.group_norm_bwd(s["x"], s["d_out"], s["weight"], **kw)
    if op == "conv_step":
        return _conv_step(s)
    if op in ("conv_fwd", "conv_bwd"):
        return _conv(s)
    if op == "scan_step":
        return _scan_step(s)
    if op in ("scan_fwd", "scan_train"):
        return _scan(s)
    return _norm(s)


# ----------------------------------------------------------------------------
# plain forms, fp32
# ----------------------------------------------------------------------------

def _dsilu(x, sg):
    return sg * (1 + x * (1 - sg))


def _sequences(s, B, T, dev):
    """Start and end of every sequence along the flattened (B T) tokens, and each token's sequence."""
    if s["cu"] is None:
        start = torch.arange(B, device=dev) * T
        return start, start + T, torch.arange(B, device=dev).repeat_interleave(T)
    cu = s["cu"].long()
    return cu[:-1], cu[1:], torch.searchsorted(cu[1:], torch.arange(B * T, device=dev), right=True)


def _conv_step(s):
    win = torch.cat([s["state"].float(), s["x"].float()[:, None]], 1)
    p = (win * s["weight"].t()).sum(1) + s["bias"]
    s["out_state"].copy_(win[:, 1:])
    return {"y": (p * torch.sigmoid(p)).to(s["x"].dtype), "state": s["out_state"]}


def _shift(x, head, pos, j, sid):
    """x_{t - j} of each token's own sequence; before its start, the last rows of `head` (zeros where it has none)."""
    y = torch.zeros_like(x)
    if j < x.shape[0]:
        y[j:] = x[:x.shape[0] - j]
    before = pos < j
    if head is None:
        return torch.where(before[:, None], torch.zeros_like(y), y)
    row = (CONV_W - 1 - j + pos).clamp(0, CONV_W - 2)
    return torch.where(before[:, None], head[sid, row], y)


def _conv(s):
    x3 = s["x"]
    B, T, D = x3.shape
    x = x3.float().reshape(B * T, D)
    w = s["weight"]
    start, end, sid = _sequences(s, B, T, x.device)
    t = torch.arange(B * T, device=x.device)
    pos = t - start[sid]
    head = None if s["h0"] is None else s["h0"].float()
    if s["op"] == "conv_fwd":
        p = s["bias"] + sum(_shift(x, head, pos, CONV_W - 1 - j, sid) * w[:, j] if j < CONV_W - 1 else x * w[:, j]
                            for j in range(CONV_W))
        y = (p * torch.sigmoid(p)).to(x3.dtype).view(B, T, D)
        # the last W - 1 inputs of each sequence, reaching into its own initial state where it is shorter
        n = (end - start)[:, None]
        at = n - (CONV_W - 1) + torch.arange(CONV_W - 1, device=x.device)
        tail = x[(start[:, None] + at).clamp(0, max(B * T - 1, 0))]
        if head is None:
            old = torch.zeros_like(tail)
        else:
            old = torch.gather(head, 1, (at + CONV_W - 1).clamp(0, CONV_W - 2)[..., None].expand(-1, -1, D))
        fs = torch.where((at < 0)[..., None], old, tail).to(x3.dtype)
        return {"y": y, "state": fs}
    dy = s["d_out"].float().reshape(B * T, D)
    taps = [_shift(x, head, pos, CONV_W - 1 - j, sid) if j < CONV_W - 1 else x for j in range(CONV_W)]
    p = s["bias"] + sum(taps[j] * w[:, j] for j in range(CONV_W))
    sg = torch.sigmoid(p)
    dp = dy * _dsilu(p, sg)
    left = end[sid] - 1 - t  # tokens of the same sequence after this one

    def ahead(j):
        z = torch.zeros_like(dp)
        if j < dp.shape[0]:
            z[:dp.shape[0] - j] = dp[j:]
        return torch.where((left < j)[:, None], torch.zeros_like(z), z)

    dx = sum((ahead(CONV_W - 1 - j) if j < CONV_W - 1 else dp) * w[:, j] for j in range(CONV_W))
    res = {"dx": dx.to(x3.dtype).view(B, T, D), "dbias": dp.sum(0),
           "dweight": torch.stack([(dp * taps[j]).sum(0) for j in range(CONV_W)], 1)}
    if head is not None:
        # state row i holds x_{i - (W - 1)}: tap j of token m reads it where i = m + j
        i = torch.arange(CONV_W - 1, device=x.device)[:, None]
        m = torch.arange(CONV_W - 1, device=x.device)[None, :]
        j = i - m
        live = (j >= 0) & (m < (end - start)[:, None, None])
        rows = dp[(start[:, None] + m).clamp(0, B * T - 1)]
        coef = torch.where(live[..., None], w.t()[j.clamp(0, CONV_W - 1)], torch.zeros((), device=x.device))
        res["d_initial_state"] = (coef * rows[:, None]).sum(2).to(x3.dtype)
    return res


def _scan_step(s):
    u, z = s["u"].float(), s["z"].float()
    per = s["D"] // s["G"]
    Bm, Cm = (s[k].float().repeat_interleave(per, 1) for k in ("Bm", "Cm"))
    raw = s["dt"].float() + s["dt_bias"]
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    h = torch.exp(dt[..., None] * s["A"]) * s["state"] + (dt * u)[..., None] * Bm
    s["out_state"].copy_(h)
    y = (h * Cm).sum(-1) + s["Dskip"] * u
    return {"y": (y * z * torch.sigmoid(z)).to(s["u"].dtype), "state": s["out_state"]}


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis by doubling; overwrites its arguments."""
    k = 1
    while k < a.shape[0]:
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _scan(s):
    u3 = s["u"]
    B, T, D = u3.shape
    G, N = s["G"], s["N"]
    M, per = B * T, D // G
    flat = lambda k: s[k].float().reshape(M, -1)  # noqa: E731
    u, z, A = flat("u"), flat("z"), s["A"]
    raw = flat("dt") + s["dt_bias"]
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    Bm, Cm = (s[k].float().reshape(M, G, 1, N).expand(M, G, per, N).reshape(M, D, N) for k in ("Bm", "Cm"))
    start, end, sid = _sequences(s, B, T, u.device)
    full = end > start
    first, last = start[full], end[full] - 1
    a = torch.exp(dt[..., None] * A)
    x = dt * u
    h = x[..., None] * Bm
    if s["h0"] is not None:
        h[first] += a[first] * s["h0"][full]
    run_a = a.clone()
    run_a[first] = 0  # nothing passes from one sequence to the next
    h = _recurrence(run_a, h)
    del run_a
    y = (h * Cm).sum(-1) + s["Dskip"] * u
    sg = torch.sigmoid(z)
    out = (y * z * sg).to(u3.dtype).view(B, T, D)
    fs = torch.zeros(start.numel(), D, N, device=u.device) if s["h0"] is None else s["h0"].clone()
    fs[full] = h[last]
    if s["op"] == "scan_fwd":
        return {"y": out, "state": fs}
    d_out = flat("d_out")
    dy = d_out * z * sg
    g = dy[..., None] * Cm
    nxt = torch.zeros_like(a)
    nxt[:-1] = a[1:]
    nxt[last] = 0
    dh = _recurrence(nxt.flip(0), g.flip(0)).flip(0)
    del nxt, g
    dC = (dy[..., None] * h).view(M, G, per, N).sum(2)
    dB = (x[..., None] * dh).view(M, G, per, N).sum(2)
    dx = (dh * Bm).sum(-1)
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    prev[first] = 0 if s["h0"] is None else s["h0"][full]
    del h
    ah = dh * a
    d0 = ah[first]
    q = ah * prev
    ddt = ((q * A).sum(-1) + u * dx) * torch.sigmoid(raw)
    res = {"du": (dt * dx + s["Dskip"] * dy).to(u3.dtype).view(B, T, D), "ddt": ddt.to(u3.dtype).view(B, T, D),
           "dz": (d_out * y * _dsilu(z, sg)).to(u3.dtype).view(B, T, D),
           "dB": dB.to(u3.dtype).view(B, T, G, N), "dC": dC.to(u3.dtype).view(B, T, G, N),
           "dA": (q * dt[..., None]).sum(0), "dD": (dy * u).sum(0), "ddt_bias": ddt.sum(0)}
    if s["h0"] is not None:
        res["d_initial_state"] = torch.zeros_like(s["h0"])
        res["d_initial_state"][full] = d0
    return {"y": out, "state": fs, **res}


def _norm(s, eps=1e-6):
    x2 = s["x"]
    rows, C = x2.shape
    g = s["groups"]
    split = lambda v: v.view(rows, g, C // g)  # noqa: E731
    x = x2.float()
    first = s["gate_first"]
    gate = None if s["gate"] is None else s["gate"].float()
    sg = None if gate is None else torch.sigmoid(gate)
    act = None if gate is None else gate * sg
    xp = x * act if first else x
    mean = split(xp).mean(-1, keepdim=True) if s["center"] else 0.0
    xc = split(xp) - mean
    r = torch.rsqrt((xc * xc).mean(-1, keepdim=True) + eps)
    n = (xc * r).view(rows, C)
    v = n * s["weight"]
    if s["bias"] is not None:
        v = v + s["bias"]
    if s["op"] == "norm_fwd":
        if gate is None:
            return (v * torch.sigmoid(v)).to(x2.dtype)
        return (v if first else v * act).to(x2.dtype)
    dy = s["d_out"].float()
    res = {}
    if gate is None:
        dv = dy * _dsilu(v, torch.sigmoid(v))
    else:
        dv = dy if first else dy * act
    if gate is not None and not first:
        res["dgate"] = (dy * v * _dsilu(gate, sg)).to(x2.dtype)
    res["dweight"] = (dv * n).sum(0)
    if s["bias"] is not None:
        res["dbias"] = dv.sum(0)
    dn, n3 = split(dv * s["weight"]), split(n)
    dx = dn - n3 * (dn * n3).mean(-1, keepdim=True)
    if s["center"]:
        dx = dx - dn.mean(-1, keepdim=True)
    dx = (r * dx).view(rows, C)
    if first:
        res["dgate"] = (dx * x * _dsilu(gate, sg)).to(x2.dtype)
        dx = dx * act
    res["dx"] = dx.to(x2.dtype)
    return res


# ----------------------------------------------------------------------------
# the definitions, fp64
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if op.startswith("norm"):
        return _norm64(f)
    if op == "conv_step":
        win = torch.cat([f["state"], f["x"][:, None]], 1)
        return {"y": torch.nn.functional.silu(torch.einsum("bwd,dw->bd", win, f["weight"]) + f["bias"]),
                "state": win[:, 1:]}
    if op.startswith("conv"):
        return _conv64(f)
    if op == "scan_step":
        f["u"], f["dt"], f["z"], f["Bm"], f["Cm"] = (f[k][:, None] for k in ("u", "dt", "z", "Bm", "Cm"))
        f["h0"], f["cu"] = f["state"], None
        r = _scan64(f)
        return {"y": r["y"][:, 0], "state": r["state"]}
    return _scan64(f)


def _norm64(f, eps=1e-6):
    leaf = {k: f[k].clone().requires_grad_() for k in ("x", "gate", "weight", "bias") if f[k] is not None}
    C = f["x"].shape[1] // f["groups"]
    silu = torch.nn.functional.silu
    x = leaf["x"] * silu(leaf["gate"]) if f["gate_first"] else leaf["x"]
    out = []
    for g in range(f["groups"]):
        cols = slice(g * C, (g + 1) * C)
        p = x[:, cols]
        if f["center"]:
            p = p - p.sum(1, keepdim=True) / C
        v = p / torch.sqrt(p.square().sum(1, keepdim=True) / C + eps) * leaf["weight"][cols]
        if "bias" in leaf:
            v = v + leaf["bias"][cols]
        if "gate" not in leaf:
            v = silu(v)
        elif not f["gate_first"]:
            v = v * silu(leaf["gate"][:, cols])
        out.append(v)
    y = torch.cat(out, 1)
    if f["op"] == "norm_fwd":
        return y.detach()
    grads = torch.autograd.grad(y, list(leaf.values()), f["d_out"])
    return {"d" + k: g for k, g in zip(leaf, grads)}


def _bounds(f, B, T):
    if f["cu"] is None:
        return [(b, 0, T) for b in range(B)]
    cu = f["cu"].tolist()
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def _conv64(f):
    B, T, D = f["x"].shape
    leaf = {k: f[k].clone().requires_grad_() for k in ("x", "weight", "bias", "h0") if f[k] is not None}
    zeros = f["x"].new_zeros(CONV_W - 1, D)
    ys, states = [], []
    for n, (b, t0, t1) in enumerate(_bounds(f, B, T)):
        x = torch.cat([leaf["h0"][n] if "h0" in leaf else zeros, leaf["x"][b, t0:t1]])
        states.append(x[x.shape[0] - (CONV_W - 1):])
        if t1 > t0:
            p = torch.einsum("tdw,dw->td", x.unfold(0, CONV_W, 1), leaf["weight"]) + leaf["bias"]
            ys.append(torch.nn.functional.silu(p))
    y = torch.cat(ys).view(B, T, D)
    if f["op"] == "conv_fwd":
        return {"y": y.detach(), "state": torch.stack(states).detach()}
    grads = torch.autograd.grad(y, list(leaf.values()), f["d_out"], allow_unused=True)
    return {{"h0": "d_initial_state"}.get(k, "d" + k): g for k, g in zip(leaf, grads)}


def _scan64(f):
    """Token by token, all sequences that have the token at once; the reverse mode likewise."""
    B, T, D = f["u"].shape
    G, N = f["G"], f["N"]
    seqs = _bounds(f, B, T)
    S, longest = len(seqs), max(t1 - t0 for _, t0, t1 in seqs)
    if S * longest * D > 1 << 26 or (f["op"] == "scan_train" and S * longest * D * N > 1 << 30):
        return None
    dev = f["u"].device
    lens = torch.tensor([t1 - t0 for _, t0, t1 in seqs], device=dev)

    def rows(v):  # (longest, S, ...): each sequence from its own start, zeros after its end
        v = v.reshape(B, T, -1)
        r = v.new_zeros(longest, S, v.shape[2])
        for n, (b, t0, t1) in enumerate(seqs):
            r[:t1 - t0, n] = v[b, t0:t1]
        return r

    def back(r, *shape):  # the inverse of rows()
        v = r.new_zeros(B, T, r.shape[2])
        for n, (b, t0, t1) in enumerate(seqs):
            v[b, t0:t1] = r[:t1 - t0, n]
        return v.view(B, T, *shape)

    u, z, raw = rows(f["u"]), rows(f["z"]), rows(f["dt"]) + f["dt_bias"]
    Bm, Cm = (rows(f[k]).view(longest, S, G, N) for k in ("Bm", "Cm"))
    dt = torch.nn.functional.softplus(raw, threshold=1e9)
    wide = lambda v: v[:, :, None].expand(S, G, D // G, N).reshape(S, D, N)  # noqa: E731
    h = f["u"].new_zeros(S, D, N) if f["h0"] is None else f["h0"].clone()
    train = f["op"] == "scan_train"
    y = torch.empty_like(u)
    past = []
    for t in range(longest):
        if train:
            past.append(h)
        live = (t < lens)[:, None, None]
        new = torch.exp(dt[t][..., None] * f["A"]) * h + (dt[t] * u[t])[..., None] * wide(Bm[t])
        h = torch.where(live, new, h)
        y[t] = (new * wide(Cm[t])).sum(-1) + f["Dskip"] * u[t]
    sil = torch.nn.functional.silu(z)
    res = {"y": back(y * sil, D), "state": h}
    if not train:
        return res
    g = rows(f["d_out"])
    sig = torch.sigmoid(z)
    dy = g * sil
    du, ddt = torch.empty_like(u), torch.empty_like(u)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    dA = torch.zeros_like(f["A"])
    dh = torch.zeros_like(h)
    part = lambda v: v.view(S, G, D // G, N).sum(2)  # noqa: E731
    for t in range(longest - 1, -1, -1):
        live = (t < lens)[:, None, None]
        a = torch.exp(dt[t][..., None] * f["A"])
        hp, x = past.pop(), dt[t] * u[t]
        now = a * hp + x[..., None] * wide(Bm[t])
        dh = torch.where(live, dh + dy[t][..., None] * wide(Cm[t]), dh)
        dC[t] = part(dy[t][..., None] * now)
        dB[t] = part(dh * x[..., None])
        dx = (dh * wide(Bm[t])).sum(-1)
        through = torch.where(live, dh * a, dh)
        q = torch.where(live, through * hp, torch.zeros_like(hp))
        dA += (q * dt[t][..., None]).sum(0)
        ddt[t] = torch.where(live[..., 0], ((q * f["A"]).sum(-1) + dx * u[t]) * torch.sigmoid(raw[t]), 0.0)
        du[t] = dx * dt[t] + f["Dskip"] * dy[t]
        dh = through
    res.update(du=back(du, D), ddt=back(ddt, D), dz=back(g * y * sig * (1 + z * (1 - sig)), D), dB=back(dB.flatten(2), G, N),
               dC=back(dC.flatten(2), G, N), dA=dA, dD=(dy * u).sum((0, 1)), ddt_bias=ddt.sum((0, 1)))
    if f["h0"] is not None:
        res["d_initial_state"] = dh
    return res


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def work(case):
    """Each input read once, each output written once; an exponential counts as one operation."""
    e, op = ELEM[case["dtype"]], case["op"]
    if op.startswith("norm"):
        n = case["rows"] * case["C"]
        if op == "norm_fwd":
            return {"bytes": n * e * (3 if case["gated"] else 2) + 4 * case["C"],
                    "flops": n * (12 if case["gated"] else 11)}
        return {"bytes": n * e * (5 if case["gated"] else 3) + 8 * case["C"], "flops": n * (26 if case["gated"] else 20)}
    D = case["D"]
    if op.startswith("conv"):
        par = 4 * D * (CONV_W + 1)
        tokens = case["B"] * case.get("T", 1)
        states = (case["B"] if op == "conv_step" else (case["nseq"] or case["B"])) * (CONV_W - 1) * D * e
        if op == "conv_bwd":
            states *= 2 if case["nseq"] else 0  # read, and its gradient written
            return {"bytes": tokens * D * e * 3 + 2 * par + states, "flops": tokens * D * (6 * CONV_W + 8)}
        states *= 2 if op == "conv_step" or case["nseq"] else 1
        return {"bytes": tokens * D * e * 2 + par + states, "flops": tokens * D * (2 * CONV_W + 5)}
    G, N = case["G"], case["N"]
    tokens = case["B"] * case.get("T", 1)
    seqs = case.get("nseq") or case["B"]
    par = 4 * D * (N + 2)
    state = 4 * seqs * D * N
    given = op == "scan_step" or bool(case["nseq"])
    if op == "scan_train":
        # forward and backward: u, dt, z, B, C and d_out in; out, du, ddt, dz, dB and dC out
        return {"bytes": tokens * e * (8 * D + 4 * G * N) + 2 * par + state * (3 if given else 1),
                "flops": tokens * D * (26 * N + 40)}
    return {"bytes": tokens * e * (4 * D + 2 * G * N) + par + state * (2 if given else 1),
            "flops": tokens * D * (7 * N + 16)}
