"""The operators of the attention layers that stand between linear-attention
layers, and of the gated recurrence that takes a linear-attention layer's
place: a gated linear recurrence, the norm and rotation of queries and keys,
and attention with a sliding window and a few first tokens that stay visible.
For each a range of sizes, a plain form in elementary torch operations (fp32
throughout, rounded once at the end), the calls a user makes of this package,
and the definition in fp64.

    rec    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t,
           log a_t = -C softplus(lam) sigmoid(r_t)                     per channel
    rope   rotate(x (mean(x^2) + eps)^-1/2 weight, position)           per head
    attn   token i sees j <= i with i - j < window or j < sinks; heads share
           keys and values in groups.  The step keeps a sequence's keys and
           values in sinks + window rows: token p in row p while p < sinks,
           in row sinks + (p - sinks) % window from there on.

A packed batch is (1, T, ...) with int32 offsets cu_seqlens.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}
RATE = 8.0
EPS = 1e-6
BASE = 10000.0


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one decoded token for 64 sequences
        {"name": "rec_step", "op": "rec_step", "B": 64, "D": 2048, "dtype": "bf16"},
        # prompts of the package's training shape
        {"name": "rec_prompt", "op": "rec_fwd", "B": 4, "T": 4096, "D": 2048, "nseq": 0, "dtype": "bf16"},
        # one long document alone: few channels, a long serial axis
        {"name": "rec_long", "op": "rec_fwd", "B": 1, "T": 65536, "D": 1024, "nseq": 0, "dtype": "bf16"},
        # a training step over packed documents: forward, then every gradient
        {"name": "rec_train", "op": "rec_train", "B": 1, "T": 16384, "D": 2048, "nseq": 12, "dtype": "bf16"},
        # one decoded token for 64 sequences, far into their texts
        {"name": "rope_decode", "op": "rope_fwd", "B": 64, "T": 1, "H": 16, "Hk": 4, "d": 128, "rot": 128,
         "pairs": "halves", "nseq": 0, "positions": True, "dtype": "bf16"},
        # prompts of the package's training shape, four query heads to a key head
        {"name": "rope_prompt", "op": "rope_fwd", "B": 4, "T": 4096, "H": 16, "Hk": 4, "d": 128, "rot": 128,
         "pairs": "halves", "nseq": 0, "positions": False, "dtype": "bf16"},
        # gradients over packed documents of odd lengths in fp32, neighbouring pairs, half of the head rotated
        {"name": "rope_backward_f32", "op": "rope_bwd", "B": 1, "T": 8191, "H": 6, "Hk": 6, "d": 64, "rot": 32,
         "pairs": "neighbours", "nseq": 9, "positions": False, "dtype": "f32"},
        # prompts of the package's training shape, a window of a quarter of them and four first tokens
        {"name": "attn_prompt", "op": "attn_fwd", "B": 4, "T": 4096, "H": 16, "Hk": 4, "d": 128, "window": 1024,
         "sinks": 4, "nseq": 0},
        # ragged packed prompts, short odd window, a key head to each query head
        {"name": "attn_packed", "op": "attn_fwd", "B": 1, "T": 5003, "H": 6, "Hk": 6, "d": 64, "window": 129,
         "sinks": 0, "nseq": 9},
        # a training step on one long document: forward, then every gradient
        {"name": "attn_train", "op": "attn_train", "B": 1, "T": 16384, "H": 16, "Hk": 4, "d": 128, "window": 2048,
         "sinks": 4, "nseq": 0},
        # one decoded token for 64 sequences, most of them past their window
        {"name": "attn_step", "op": "attn_step", "B": 64, "H": 16, "Hk": 4, "d": 128, "window": 1024, "sinks": 4},
        # one decoded token of a single sequence over a long window, one key head
        {"name": "attn_step_one", "op": "attn_step", "B": 1, "H": 8, "Hk": 1, "d": 128, "window": 16384, "sinks": 4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _width(rng, lo, hi):
    """A channel count: often a multiple of 64, else anything."""
    d = _log(rng, lo, hi)
    return max(64, d // 64 * 64) if rng.random() < 0.6 else d


def _tokens(rng, case, most):
    """B, T and the number of packed sequences of up to `most` tokens in all."""
    tokens = _log(rng, 1, max(1, min(65536, most)))
    if rng.random() < 0.4 and tokens > 8:
        case.update(B=1, T=tokens, nseq=_log(rng, 1, min(64, tokens // 4)))
    else:
        B = _log(rng, 1, min(16, tokens))
        case.update(B=B, T=tokens // B, nseq=0)
    return case


def draw(rng):
    op = rng.choice(["rec_step", "rec_fwd", "rec_fwd", "rec_train", "rope_fwd", "rope_fwd", "rope_bwd", "attn_fwd",
                     "attn_fwd", "attn_train", "attn_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rec_step":
        return {"op": op, "B": _log(rng, 1, 1024), "D": _width(rng, 64, 8192), "dtype": dtype}
    if op.startswith("rec"):
        D = _width(rng, 64, 4096)
        most = (1 << (26 if op == "rec_fwd" else 25)) // (1 if dtype == "bf16" else 2)
        return _tokens(rng, {"op": op, "D": D, "dtype": dtype}, most // D)
    Hk = rng.choice([1, 2, 3, 4, 8])
    H = Hk * rng.choice([1, 1, 2, 4, 5, 8])
    if op.startswith("rope"):
        d = rng.choice([64, 128, 128, 256])
        case = {"op": op, "H": H, "Hk": Hk, "d": d, "rot": d // rng.choice([1, 1, 2, 4]),
                "pairs": rng.choice(["halves", "neighbours"]), "positions": rng.random() < 0.5, "dtype": dtype}
        most = (1 << 25) // (1 if dtype == "bf16" else 2)
        return _tokens(rng, case, most // ((H + Hk) * d))
    d = rng.choice([64, 128])
    case = {"op": op, "H": H, "Hk": Hk, "d": d, "window": _log(rng, 1, 16384), "sinks": rng.choice([0, 0, 1, 4, 16, 64])}
    if op == "attn_step":
        rows = (1 << 26) // (Hk * d)
        case["window"] = min(case["window"], rows // 2)
        case["B"] = _log(rng, 1, min(512, rows // (case["window"] + case["sinks"])))
        return case
    # as many pairs of tokens and channels as the listed cases of the kind, at most
    most = (1 << 36) if op == "attn_fwd" else (1 << 35)
    _tokens(rng, case, min(16384, (1 << 25) // ((H + Hk) * d)))
    seen = min(case["window"] + case["sinks"], case["T"])
    while case["B"] * case["T"] * seen * H * d > most:
        case["B"], case["T"] = max(1, case["B"] // 2), max(1, case["T"] * 2 // 3)
        case["nseq"] = min(case["nseq"], case["T"])
        seen = min(case["window"] + case["sinks"], case["T"])
    return case


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _offsets(case):
    """Offsets of the case's ragged sequences (some may hold one token or none)."""
    T, nseq = case["T"], case["nseq"]
    rng = random.Random(1000003 * T + nseq)
    return [0] + sorted(rng.randint(0, T) for _ in range(nseq - 1)) + [T]


def _lengths(case):
    """Tokens each decoded sequence has behind it: most are past the window, some are new."""
    rows = case["sinks"] + case["window"]
    rng = random.Random(1000003 * rows + case["B"])
    return [rng.randint(0, rows) if rng.random() < 0.25 else rng.randint(rows, 4 * rows) for _ in range(case["B"])]


def _seqs(case):
    """(batch row, first token, end) of every sequence."""
    if not case.get("nseq"):
        return [(b, 0, case["T"]) for b in range(case["B"])]
    cu = _offsets(case)
    return [(0, a, b) for a, b in zip(cu[:-1], cu[1:])]


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op = case["op"]
    dtype = DTYPES[case.get("dtype", "bf16")]

    def normal(*shape, scale=1.0, to=dtype):
        return (torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32) * scale).to(to)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32) * (hi - lo) + lo

    s = dict(case)
    s["cu"] = None
    if case.get("nseq"):
        s["cu"] = torch.tensor(_offsets(case), dtype=torch.int32, device=dev)
    if op.startswith("rec"):
        D = case["D"]
        # decays between 0.9 and 0.999 at an open gate, as trained models start from
        decay = uniform(0.9, 0.999, D)
        s["lam"] = torch.log(torch.expm1(-torch.log(decay) / RATE))
        if op == "rec_step":
            s["x"] = normal(case["B"], D)
            gates = normal(case["B"], 2 * D)
            s["state"] = normal(case["B"], D, scale=0.5, to=torch.float32)
            s["out_state"] = torch.empty_like(s["state"])
        else:
            s["x"] = normal(case["B"], case["T"], D)
            gates = normal(case["B"], case["T"], 2 * D)  # both gates from one projection
            s["h0"] = normal(case["nseq"], D, scale=0.5, to=torch.float32) if case["nseq"] else None
            if op == "rec_train":
                s["d_out"] = normal(case["B"], case["T"], D)
        s["r"], s["i"] = gates[..., :D], gates[..., D:]
        return s
    H, Hk, d = case["H"], case["Hk"], case["d"]
    if op.startswith("rope"):
        B, T = case["B"], case["T"]
        qkv = normal(B, T, (H + 2 * Hk) * d)  # one projection's queries, keys and values
        s["q"] = qkv[..., :H * d].unflatten(-1, (H, d))
        s["k"] = qkv[..., H * d:(H + Hk) * d].unflatten(-1, (Hk, d))
        s["q_weight"], s["k_weight"] = uniform(0.5, 1.5, d), uniform(0.5, 1.5, d)
        s["inv_freq"] = BASE ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float32) / case["rot"])
        s["pos"] = None
        if case["positions"]:  # decoded or cached tokens: anywhere in texts of up to a million tokens
            start = torch.randint(0, 1 << 20, (B, 1), generator=gen, device=dev, dtype=torch.int32)
            s["pos"] = start + torch.arange(T, device=dev, dtype=torch.int32)
        if op == "rope_bwd":
            s["dq_out"], s["dk_out"] = normal(B, T, H, d), normal(B, T, Hk, d)
        return s
    if op == "attn_step":
        B, rows = case["B"], case["sinks"] + case["window"]
        s["q"] = normal(B, H, d)
        s["k"] = normal(B, Hk, d)
        s["v"] = normal(B, (H + 2 * Hk) * d)[:, (H + Hk) * d:].unflatten(-1, (Hk, d))
        s["k_cache"], s["v_cache"] = normal(B, rows, Hk, d), normal(B, rows, Hk, d)
        s["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
        return s
    B, T = case["B"], case["T"]
    s["q"], s["k"] = normal(B, T, H, d), normal(B, T, Hk, d)  # normed and rotated
    # values where the projection left them, behind its queries and keys
    s["v"] = normal(B, T, (H + 2 * Hk) * d)[..., (H + Hk) * d:].unflatten(-1, (Hk, d))
    if op == "attn_train":
        s["d_out"] = normal(B, T, H, d)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        from linear_attention_sequence_chunked_gb300 import attention, mixer
        if op == "rec_step":
            y = mixer.gated_scan_step(s["x"], s["r"], s["i"], s["lam"], s["state"], rate=RATE, out_state=s["out_state"])
            return {"y": y, "state": s["out_state"]}
        if op == "rec_fwd":
            y, fs = mixer.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], rate=RATE, initial_state=s["h0"],
                                         cu_seqlens=s["cu"])
            return {"y": y, "state": fs}
        if op == "rec_train":
            kw = dict(rate=RATE, initial_state=s["h0"], cu_seqlens=s["cu"])
            y, fs, saved = mixer.gated_scan_fwd(s["x"], s["r"], s["i"], s["lam"], save_for_backward=True, **kw)
            g = mixer.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["d_out"], saved, **kw)
            return {"y": y, "state": fs, **g}
        if op.startswith("rope"):
            kw = dict(inv_freq=s["inv_freq"], positions=s["pos"], cu_seqlens=s["cu"], eps=EPS,
                      interleaved=s["pairs"] == "neighbours")
            if op == "rope_fwd":
                q, k = attention.qk_norm_rope_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], **kw)
                return {"q": q, "k": k}
            return attention.qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["q_weight"], s["k_weight"],
                                              **kw)
        if op == "attn_step":
            out = attention.window_attention_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["lengths"],
                                                  sinks=s["sinks"])
            return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        kw = dict(window=s["window"], sinks=s["sinks"], cu_seqlens=s["cu"])
        if op == "attn_fwd":
            return attention.window_attention_fwd(s["q"], s["k"], s["v"], **kw)
        out, lse = attention.window_attention_fwd(s["q"], s["k"], s["v"], save_for_backward=True, **kw)
        g = attention.window_attention_bwd(s["q"], s["k"], s["v"], out, lse, s["d_out"], **kw)
        return {"out": out, **g}
    if op == "rec_step":
        return _rec_step(s)
    if op.startswith("rec"):
        return _rec(s)
    if op.startswith("rope"):
        return _rope(s)
    if op == "attn_step":
        return _attn_step(s)
    return _attn(s)


# ----------------------------------------------------------------------------
# plain forms, fp32
# ----------------------------------------------------------------------------

def _gates(s):
    sr, si = torch.sigmoid(s["r"].float()), torch.sigmoid(s["i"].float())
    lam = s["lam"]
    sp = torch.clamp(lam, min=0) + torch.log1p(torch.exp(-lam.abs()))
    la = -RATE * sp * sr
    return sr, si, la, torch.exp(la), torch.sqrt(-torch.expm1(2 * la))


def _rec_step(s):
    x = s["x"].float()
    _, si, _, a, m = _gates(s)
    h = a * s["state"] + m * (si * x)
    s["out_state"].copy_(h)
    return {"y": h.to(s["x"].dtype), "state": s["out_state"]}


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along the first axis by doubling; overwrites its arguments."""
    k = 1
    while k < a.shape[0]:
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _rec(s):
    x3 = s["x"]
    B, T, D = x3.shape
    dev = x3.device
    x = x3.float().reshape(B * T, D)
    sr, si, la, a, m = (v.reshape(B * T, D) for v in _gates(s))
    if s["cu"] is None:
        start = torch.arange(B, device=dev) * T
        end = start + T
    else:
        cu = s["cu"].long()
        start, end = cu[:-1], cu[1:]
    full = end > start
    first, last = start[full], end[full] - 1
    gx = si * x
    h = m * gx
    if s["h0"] is not None:
        h[first] += a[first] * s["h0"][full]
    run_a = a.clone()
    run_a[first] = 0  # nothing passes from one sequence to the next
    h = _recurrence(run_a, h)
    del run_a
    fs = torch.zeros(start.numel(), D, device=dev) if s["h0"] is None else s["h0"].clone()
    fs[full] = h[last]
    res = {"y": h.to(x3.dtype).view(B, T, D), "state": fs}
    if s["op"] == "rec_fwd":
        return res
    nxt = torch.zeros_like(a)
    nxt[:-1] = a[1:]
    nxt[last] = 0
    dh = _recurrence(nxt.flip(0), s["d_out"].float().reshape(B * T, D).flip(0)).flip(0)
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    prev[first] = 0 if s["h0"] is None else s["h0"][full]
    dgx = dh * m
    through = torch.where(m > 0, a * a / m, torch.zeros_like(m))
    dla = dh * (a * prev - through * gx)
    to = lambda v: v.to(x3.dtype).view(B, T, D)  # noqa: E731
    res.update(dx=to(dgx * si), di=to(dgx * x * si * (1 - si)), dr=to(dla * la * (1 - sr)),
               dlam=((dla * sr).sum(0, dtype=torch.float64) * (-RATE * torch.sigmoid(s["lam"]))).float())
    if s["h0"] is not None:
        res["d_initial_state"] = torch.zeros_like(s["h0"])
        res["d_initial_state"][full] = dh[first] * a[first]
    return res


def _positions(s):
    B, T = s["q"].shape[:2]
    if s["pos"] is not None:
        return s["pos"].long()
    t = torch.arange(T, device=s["q"].device)
    if s["cu"] is None:
        return t.expand(B, T)
    cu = s["cu"].long()
    return (t - cu[torch.searchsorted(cu[1:], t, right=True)])[None]


def _turn(x, cos, sin, rot, pairs):
    """The first `rot` channels of each head turned by the angles of their pairs."""
    head = x[..., :rot]
    out = x.clone()
    if pairs == "halves":
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return out


def _rope(s):
    angle = _positions(s).double()[..., None, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    res = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_weight"]
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        if s["op"] == "rope_fwd":
            res[n] = _turn(x * r * w, cos, sin, s["rot"], s["pairs"]).to(s[n].dtype)
            continue
        g = _turn(s[f"d{n}_out"].float(), cos, -sin, s["rot"], s["pairs"])
        nx = x * r
        gw = g * w
        res["d" + n] = (r * (gw - nx * (gw * nx).mean(-1, keepdim=True))).to(s[n].dtype)
        res[f"d{n}_weight"] = (g * nx).flatten(0, -2).sum(0, dtype=torch.float64).float()
    return res


def _seen(s, i0, i1, lo, dev):
    """Keys that the queries [i0, i1) look at, and which of them each one sees."""
    first = min(s["sinks"], lo)
    j = torch.cat([torch.arange(first, device=dev), torch.arange(lo, i1, device=dev)])
    i = torch.arange(i0, i1, device=dev)[:, None]
    return j, (j <= i) & ((i - j < s["window"]) | (j < s["sinks"]))


BLOCK = 512


def _attn(s):
    q3, k3, v3 = s["q"], s["k"], s["v"]
    B, T, H, d = q3.shape
    Hk = k3.shape[2]
    G, scale, dev = H // Hk, d ** -0.5, q3.device
    train = s["op"] == "attn_train"
    out = torch.empty(B, T, H, d, device=dev)
    if train:
        dq = torch.empty_like(out)
        dk, dv = (torch.zeros(B, T, Hk, d, device=dev) for _ in range(2))
    seqs = [(slice(0, B), 0, T)] if s["cu"] is None else [(slice(0, 1), a, b) for _, a, b in _seqs(s)]
    for rows, t0, t1 in seqs:
        heads = lambda v: v[rows, t0:t1].float().unflatten(2, (Hk, -1)).permute(0, 2, 3, 1, 4)  # noqa: E731
        q, k, v = heads(q3), heads(k3)[:, :, 0], heads(v3)[:, :, 0]
        g = heads(s["d_out"]) if train else None
        for i0 in range(0, t1 - t0, BLOCK):
            i1 = min(i0 + BLOCK, t1 - t0)
            j, mask = _seen(s, i0, i1, max(0, i0 - s["window"] + 1), dev)
            kj, vj = k[:, :, j], v[:, :, j]
            qi = q[:, :, :, i0:i1].flatten(2, 3)
            S = (qi @ kj.transpose(-1, -2)).unflatten(2, (G, -1)) * scale
            S = torch.where(mask, S, torch.full((), -math.inf, device=dev))
            e = torch.exp(S - S.amax(-1, keepdim=True))
            P = (e / e.sum(-1, keepdim=True)).flatten(2, 3)
            o = P @ vj
            put = lambda v: v.unflatten(2, (G, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # noqa: E731
            out[rows, t0 + i0:t0 + i1] = put(o)
            if train:
                do = g[:, :, :, i0:i1].flatten(2, 3)
                dP = do @ vj.transpose(-1, -2)
                dS = P * (dP - (do * o).sum(-1, keepdim=True)) * scale
                dq[rows, t0 + i0:t0 + i1] = put(dS @ kj)
                dk[rows, t0 + j] += (dS.transpose(-1, -2) @ qi).permute(0, 2, 1, 3)
                dv[rows, t0 + j] += (P.transpose(-1, -2) @ do).permute(0, 2, 1, 3)
    if not train:
        return out.to(q3.dtype)
    return {"out": out.to(q3.dtype), "dq": dq.to(q3.dtype), "dk": dk.to(q3.dtype), "dv": dv.to(q3.dtype)}


def _attn_step(s):
    q, kc, vc = s["q"].float(), s["k_cache"], s["v_cache"]
    B, H, d = q.shape
    R, Hk = kc.shape[1:3]
    p = s["lengths"].long()
    row = torch.where(p < s["sinks"], p, s["sinks"] + (p - s["sinks"]) % s["window"])
    b = torch.arange(B, device=q.device)
    kc[b, row] = s["k"]
    vc[b, row] = s["v"]
    live = torch.arange(R, device=q.device) <= p[:, None]
    k, v = kc.float().transpose(1, 2), vc.float().transpose(1, 2)
    S = q.unflatten(1, (Hk, -1)) @ k.transpose(-1, -2) * d ** -0.5
    S = torch.where(live[:, None, None], S, torch.full((), -math.inf, device=q.device))
    e = torch.exp(S - S.amax(-1, keepdim=True))
    out = (e @ v) / e.sum(-1, keepdim=True)
    return {"out": out.flatten(1, 2).to(s["q"].dtype), "k_cache": kc, "v_cache": vc}


# ----------------------------------------------------------------------------
# the definitions, fp64
# ----------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    op = case["op"]
    if op.startswith("rec"):
        return _rec64(f)
    if op.startswith("rope"):
        return _rope64(f)
    if op == "attn_step":
        return _step64(f)
    return _attn64(f)


def _decay64(f, leaf):
    """The decay a and the input b of every token."""
    gate = torch.nn.functional.logsigmoid(leaf["r"]).exp()
    la = -RATE * torch.nn.functional.softplus(leaf["lam"], threshold=1e9) * gate
    return la.exp(), torch.sqrt(1 - (2 * la).exp()) * torch.sigmoid(leaf["i"]) * leaf["x"]


def _rec64(f):
    leaf = {k: f[k].clone().requires_grad_() for k in ("x", "r", "i", "lam")}
    a, b = _decay64(f, leaf)
    if f["op"] == "rec_step":
        h = (a * f["state"] + b).detach()
        return {"y": h, "state": h}
    B, T, D = f["x"].shape
    seqs = _seqs(f)
    h0 = f["h0"] if f["h0"] is not None else f["x"].new_zeros(len(seqs), D)
    ad, bd = a.detach(), b.detach()
    train = f["op"] == "rec_train"
    y, prev, dh = torch.empty_like(ad), torch.empty_like(ad), torch.empty_like(ad)
    fs, d0 = h0.clone(), torch.zeros_like(h0)
    # dense rows step together, packed sequences one by one
    groups = [(slice(0, B), slice(0, B), 0, T)] if f["cu"] is None else \
        [(slice(0, 1), slice(n, n + 1), t0, t1) for n, (_, t0, t1) in enumerate(seqs)]
    for rows, n, t0, t1 in groups:
        h = h0[n]
        for t in range(t0, t1):
            if train:
                prev[rows, t] = h
            h = torch.addcmul(bd[rows, t], ad[rows, t], h, out=y[rows, t])
        fs[n] = h
        if train:
            back = torch.zeros_like(h)
            for t in range(t1 - 1, t0 - 1, -1):
                torch.add(f["d_out"][rows, t], back, out=dh[rows, t])
                back = ad[rows, t] * dh[rows, t]
            d0[n] = back
    res = {"y": y, "state": fs}
    if train:
        grads = torch.autograd.grad((a, b), list(leaf.values()), (dh * prev, dh))
        res.update({"d" + k: g for k, g in zip(leaf, grads)})
        if f["h0"] is not None:
            res["d_initial_state"] = d0
    return res


def _rope64(f):
    B, T = f["q"].shape[:2]
    pos = f["pos"]
    if pos is None:
        pos = torch.cat([torch.arange(t1 - t0, device=f["q"].device) for _, t0, t1 in _seqs(f)]).view(B, T)
    rot = f["rot"]
    unit = torch.polar(torch.ones((), dtype=torch.float64, device=pos.device).expand(B, T, 1, rot // 2),
                       pos.double()[:, :, None, None] * f["inv_freq"])
    res = {}
    for n in ("q", "k"):
        x, w = (f[m].clone().requires_grad_() for m in (n, n + "_weight"))
        v = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w
        part = v[..., :rot]
        if f["pairs"] == "halves":
            z = torch.complex(*part.chunk(2, -1)) * unit
            turned = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.complex(*part.unflatten(-1, (rot // 2, 2)).unbind(-1)) * unit
            turned = torch.stack([z.real, z.imag], -1).flatten(-2)
        y = torch.cat([turned, v[..., rot:]], -1)
        if f["op"] == "rope_fwd":
            res[n] = y.detach()
        else:
            res["d" + n], res[f"d{n}_weight"] = torch.autograd.grad(y, (x, w), f[f"d{n}_out"])
    return res


def _attn64(f):
    """Head by head, a stretch of queries at a time, gradients by autograd."""
    B, T, H, d = f["q"].shape
    Hk = f["k"].shape[2]
    G, dev, W, S = H // Hk, f["q"].device, f["window"], f["sinks"]
    train = f["op"] == "attn_train"
    out = torch.empty_like(f["q"])
    grads = {n: torch.zeros_like(f[n], memory_format=torch.contiguous_format) for n in ("q", "k", "v")}
    step = 1024
    for b, t0, t1 in _seqs(f):
        for i0 in range(t0, t1, step):
            i1 = min(i0 + step, t1)
            cols = torch.unique(torch.cat([torch.arange(t0, min(t0 + S, i1)),
                                           torch.arange(max(t0, i0 + 1 - W), i1)])).to(dev)
            far = torch.arange(i0, i1, device=dev)[:, None] - cols
            hidden = (far < 0) | ((far >= W) & (cols >= t0 + S))
            for h in range(Hk):
                leaf = [f["q"][b, i0:i1, h * G:(h + 1) * G].clone(), f["k"][b, cols, h], f["v"][b, cols, h]]
                if train:
                    leaf = [x.requires_grad_() for x in leaf]
                logits = torch.einsum("igd,jd->gij", leaf[0], leaf[1]) / math.sqrt(d)
                o = torch.einsum("gij,jd->igd", torch.softmax(logits.masked_fill(hidden, -math.inf), -1), leaf[2])
                out[b, i0:i1, h * G:(h + 1) * G] = o.detach()
                if train:
                    gq, gk, gv = torch.autograd.grad(o, leaf, f["d_out"][b, i0:i1, h * G:(h + 1) * G])
                    grads["q"][b, i0:i1, h * G:(h + 1) * G] = gq
                    grads["k"][b, :, h].index_add_(0, cols, gk)
                    grads["v"][b, :, h].index_add_(0, cols, gv)
    if not train:
        return out
    return {"out": out, **{"d" + n: g for n, g in grads.items()}}


def _step64(f):
    """Row by row, the cache put back into the order of its tokens."""
    q, kc, vc = f["q"], f["k_cache"].clone(), f["v_cache"].clone()
    Hk, d = kc.shape[2:]
    W, S = f["window"], f["sinks"]
    out = torch.empty_like(q)
    for b, p in enumerate(f["lengths"].tolist()):
        at = [*range(min(S, p + 1)), *(S + (j - S) % W for j in range(max(S, p - W + 1), p + 1))]
        kc[b, at[-1]], vc[b, at[-1]] = f["k"][b], f["v"][b]
        at = torch.tensor(at, device=q.device)
        w = torch.softmax(torch.einsum("hgd,jhd->hgj", q[b].unflatten(0, (Hk, -1)), kc[b, at]) / math.sqrt(d), -1)
        out[b] = torch.einsum("hgj,jhd->hgd", w, vc[b, at]).flatten(0, 1)
    return {"out": out, "k_cache": kc, "v_cache": vc}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------

def _pairs(case):
    """Pairs of a query and a key that it sees, of one head."""
    W, S, total = case["window"], case["sinks"], 0
    for _, t0, t1 in _seqs(case):
        n = t1 - t0
        near = min(n, W)
        total += near * (near + 1) // 2 + (n - near) * W
        # tokens W and later also see the first ones that the window has left
        out = max(0, n - W)
        first = min(S, out)
        total += first * (first + 1) // 2 + (out - first) * S if S else 0
    return total


def work(case):
    """Each input read once, each output written once; an exponential counts as one operation."""
    op, e = case["op"], ELEM[case.get("dtype", "bf16")]
    if op.startswith("rec"):
        D = case["D"]
        tokens = case["B"] * case.get("T", 1)
        seqs = case.get("nseq") or case["B"]
        given = op == "rec_step" or bool(case["nseq"])
        states = 4 * seqs * D * (2 if given else 1)
        if op == "rec_train":
            # x, r, i and d_out in; the output, dx, dr and di out; lam, its gradient and the initial state's
            return {"bytes": tokens * D * e * 8 + 8 * D + states + (4 * seqs * D if given else 0),
                    "flops": tokens * D * 50}
        return {"bytes": tokens * D * e * 4 + 4 * D + states, "flops": tokens * D * 17}
    H, Hk, d = case["H"], case["Hk"], case["d"]
    if op.startswith("rope"):
        tokens = case["B"] * case["T"]
        n = tokens * (H + Hk) * d
        small = 4 * (2 * d + case["rot"] // 2) + (4 * tokens if case["positions"] else 0)
        if op == "rope_fwd":
            return {"bytes": 2 * n * e + small, "flops": 7 * n}
        return {"bytes": 3 * n * e + small + 8 * d, "flops": 14 * n}
    if op == "attn_step":
        rows = sum(min(p + 1, case["sinks"] + case["window"]) for p in _lengths(case))
        # the rows that each sequence has, its new one written and not read
        return {"bytes": 2 * e * Hk * d * rows + 2 * e * case["B"] * (H + Hk) * d + 4 * case["B"],
                "flops": 4 * rows * H * d}
    tokens = case["B"] * case["T"]
    pairs = _pairs(case) * H * d
    if op == "attn_fwd":
        return {"bytes": 2 * tokens * (H + Hk) * d * e, "flops": 4 * pairs}
    # q, k, v and d_out in; out, dq, dk and dv out
    return {"bytes": 4 * tokens * (H + Hk) * d * e, "flops": 14 * pairs}
