"""The attention operators against their fp64 definitions.

Tolerances (relative L2 of a tensor), fixed before the first run.
- bf16 outputs carry one rounding: 3e-3, this package's bound for them, and the
  rounding itself (2^-8) below 16 values.
- fp32 norms and rotations: sums of up to 256 squares, an rsqrt of 2 ulp, and
  angles to 2^-28 turns (2^-25.3 radians) with two roundings behind them: 2e-6
  (about 30 x 2^-24).  Their weights' gradients are sums over all rows that may
  cancel: 1e-5.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import attention, gdn  # noqa: E402
from oracle import attention as A  # noqa: E402
from oracle import metrics  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL_BF16, TOL_F32, TOL_PAR = 3e-3, 2e-6, 1e-5


def _dev(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda").to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _round(a, dtype):
    return _np(torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype))


def _close(got, want, tol, what):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    if np.abs(want).max(initial=0.0) == 0.0:
        assert np.abs(got).max(initial=0.0) == 0.0, what
        return
    if tol == TOL_BF16 and want.size < 16:
        tol = 2.0 ** -8 + TOL_F32
    e = metrics.rel_l2(got, want)
    assert e <= tol, f"{what}: rel L2 {e:.3e} > {tol:.1e}"


def _ints(a):
    return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


# ------------------------------------------------------- norm and rotation

ROPE = [  # B, T, H, Hk, d, frequencies, neighbouring pairs, cu, far positions, slices, weights
    (1, 1, 1, 1, 32, 16, False, None, False, False, True),
    (2, 0, 4, 2, 64, 32, False, None, False, False, True),
    (2, 33, 4, 2, 64, 32, False, None, False, True, True),
    (3, 7, 5, 1, 128, 64, True, None, True, False, True),      # an odd number of heads
    (1, 77, 3, 3, 256, 128, False, [0, 0, 40, 41, 77], False, False, True),
    (1, 200, 8, 2, 128, 32, False, None, True, True, False),   # half of a head turns, no weights
    (2, 9, 2, 2, 64, 4, True, None, False, True, True),        # one lane of a row turns
    (1, 1300, 16, 4, 64, 0, False, None, False, False, True),  # the norm alone
    (1, 3001, 1, 1, 32, 12, True, [0, 3001], True, False, True),
]


def _rope_inputs(case, dtype):
    B, T, H, Hk, d, n, nxt, cu, far, sliced, weights = case
    rng = np.random.default_rng(T + H + d)
    a = dict(q=_round(rng.standard_normal((B, T, H, d)), dtype), k=_round(rng.standard_normal((B, T, Hk, d)), dtype),
             gq=_round(rng.standard_normal((B, T, H, d)), dtype), gk=_round(rng.standard_normal((B, T, Hk, d)), dtype),
             qw=_round(rng.uniform(0.5, 1.5, d), F32) if weights else None,
             kw=_round(rng.uniform(0.5, 1.5, d), F32) if weights else None,
             f=np.float32(10000.0) ** (-np.arange(n, dtype=np.float32) / max(n, 1)) if n else None)
    pos = rng.integers(-2 ** 31, 2 ** 31, (B, T)) if far else None
    t = {k: None if v is None else _dev(v, dtype if k in ("q", "k", "gq", "gk") else F32) for k, v in a.items()}
    if sliced:  # rows of a wider projection, at an odd offset
        wide = torch.full((B, T, 1 + (H + Hk) * d), float("nan"), dtype=dtype, device="cuda")
        wide[..., 1:1 + H * d], wide[..., 1 + H * d:] = t["q"].flatten(2), t["k"].flatten(2)
        t["q"], t["k"] = wide[..., 1:1 + H * d].unflatten(2, (H, d)), wide[..., 1 + H * d:].unflatten(2, (Hk, d))
    a["pos"] = A.positions_of(a["q"], cu) if pos is None else pos
    kw = dict(q_weight=t["qw"], k_weight=t["kw"], inv_freq=t["f"], positions=_ints(pos), cu_seqlens=_ints(cu),
              interleaved=nxt)
    return a, t, kw


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(map(str, c[:6])))
def test_norm_and_rotation(case, dtype):
    a, t, kw = _rope_inputs(case, dtype)
    io = TOL_BF16 if dtype == BF else TOL_F32
    q, k = attention.qk_norm_rope_fwd(t["q"], t["k"], **kw)
    for got, x, w in ((q, a["q"], a["qw"]), (k, a["k"], a["kw"])):
        _close(got, A.rope_fwd(x, w, a["f"], a["pos"], interleaved=case[6]), io, "forward")
    r = attention.qk_norm_rope_bwd(t["q"], t["k"], t["gq"], t["gk"], **kw)
    assert set(r) == ({"dq", "dk", "dq_weight", "dk_weight"} if case[10] else {"dq", "dk"})
    for n, x, w, g in (("q", a["q"], a["qw"], a["gq"]), ("k", a["k"], a["kw"], a["gk"])):
        dx, dw = A.rope_bwd(x, w, a["f"], a["pos"], g, interleaved=case[6])
        _close(r["d" + n], dx, io, "d" + n)
        if w is not None:
            _close(r[f"d{n}_weight"], dw, TOL_PAR, f"d{n}_weight")
    assert gdn.gdn_get_last_device_error() == 0


def test_far_positions_keep_their_angles():
    """A unit pair at every power of two and its neighbours: the angle itself."""
    pos = np.unique(np.concatenate([[s * (2 ** e + o) for s in (1, -1) for o in (-1, 0, 1)] for e in range(31)]))
    f = np.array([1.0, 0.3, 1e-3, 6.5, 2.0 ** -20, 100.25, 1e-12, 0.0], dtype=np.float32)
    x = np.zeros((1, len(pos), 1, 32))
    x[..., :8] = 1
    q, _ = attention.qk_norm_rope_fwd(_dev(x), _dev(x), inv_freq=_dev(f), positions=_ints(pos[None]), eps=0.0)
    angle = A._angles(pos[None], f)
    want = np.concatenate([np.cos(angle), np.sin(angle)], -1) * 2  # the rms of 8 ones in 32 is 1/2
    assert np.abs(_np(q)[..., :16] - want).max() <= 2 * (2.0 ** -25.3 + 4 * 2.0 ** -24)


def test_norm_and_rotation_autograd():
    case = (2, 19, 4, 2, 64, 16, False, None, False, True, True)
    a, t, kw = _rope_inputs(case, F32)
    leaves = [t["q"].clone().requires_grad_(), t["k"].clone().requires_grad_(), kw["q_weight"].requires_grad_(),
              kw["k_weight"].requires_grad_()]
    q, k = attention.qk_norm_rope(leaves[0], leaves[1], **kw)
    (q * t["gq"]).sum().add((k * t["gk"]).sum()).backward()
    rng = np.random.default_rng(2)
    for n, x, w, g, lx, lw in (("q", a["q"], a["qw"], a["gq"], leaves[0], leaves[2]),
                               ("k", a["k"], a["kw"], a["gk"], leaves[1], leaves[3])):
        for at, leaf in ((0, lx), (1, lw)):
            way, h = rng.standard_normal(leaf.shape), 1e-5
            ends = [(A.rope_fwd(x + (s * h * way if at == 0 else 0), w + (s * h * way if at else 0), a["f"], a["pos"])
                     * g).sum() for s in (1, -1)]
            slope = (ends[0] - ends[1]) / (2 * h)
            size = float(np.abs(_np(leaf.grad) * way).sum())
            assert abs(float((_np(leaf.grad) * way).sum()) - slope) <= 1e-5 * size + 1e-7 * abs(slope), (n, at)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        y, _ = attention.qk_norm_rope(leaves[0], leaves[1], **kw)
        d, = torch.autograd.grad(y.sum(), leaves[0], create_graph=True)
        d.sum().backward()


def test_a_bad_row_stays_alone():
    case = (2, 40, 4, 2, 64, 32, False, None, False, False, True)
    a, t, kw = _rope_inputs(case, BF)
    good = attention.qk_norm_rope_fwd(t["q"], t["k"], **kw)[0]
    t["q"][1, 3, 2, 5], t["q"][0, 0, 0, 63] = float("nan"), float("inf")
    q = attention.qk_norm_rope_fwd(t["q"], t["k"], **kw)[0]
    same = torch.ones(2, 40, 4, dtype=torch.bool, device="cuda")
    same[1, 3, 2] = same[0, 0, 0] = False
    assert torch.equal(q[same], good[same]) and torch.isnan(q[1, 3, 2]).all()


# ------------------------------------------------------------------- window
#
# Tolerances of the attention, from its roundings.  P and dS are bf16 operands:
# each element is off by at most 2^-8 of itself, uniformly distributed, so by
# about 2^-8 / sqrt(3) x 0.72 in L2 (1.65e-3, as for a bf16 output); summed over
# keys in random directions the relative error of a sum of like terms stays that
# of one term, 1.65e-3, and where terms cancel it grows against the sum.  Over
# iid values the L2 of the sum and of its terms agree, so an output carries
# sqrt(2) x 1.65e-3 = 2.4e-3 with its own rounding, within the 3e-3 of bf16
# outputs here.  Gradients of dS carry P's, dS's and the saved output's rounding
# (delta): sqrt(3) x 1.65e-3 and the final one, 3.3e-3, within this package's
# bound for gradients, 5e-3.
TOL_GRAD = 5e-3

WINDOW = [  # B, T, H, Hk, d, window, sinks, cu
    (1, 1, 1, 1, 64, 1, 0, None),
    (2, 0, 2, 1, 64, 4, 1, None),
    (1, 3, 2, 2, 128, 100, 4, None),          # shorter than everything
    (2, 127, 4, 2, 64, 1, 0, None),           # each token sees itself alone
    (2, 129, 4, 1, 128, 128, 0, None),
    (1, 128, 3, 1, 64, 17, 3, None),          # an odd group
    (1, 300, 5, 5, 128, 129, 0, None),        # a key head to each query head
    (1, 513, 2, 2, 64, 64, 128, None),        # as many first tokens as there may be
    (1, 700, 6, 2, 128, 130, 33, None),
    (2, 1000, 4, 2, 64, 1000, 5, None),       # the window is everything
    (1, 1200, 8, 1, 128, 300, 4, None),
    (1, 600, 4, 2, 128, 50, 2, [0, 0, 1, 3, 130, 131, 400, 600]),
    (1, 900, 3, 3, 64, 200, 64, [0, 256, 512, 640, 900]),
    (1, 300, 2, 1, 64, 7, 1, [0, 300]),
    (1, 130, 2, 2, 64, 9, 9, list(range(131))),  # a token each
]


def _window_inputs(case, seed=0):
    B, T, H, Hk, d, W, S, cu = case
    rng = np.random.default_rng(T + H + W + seed)
    a = {n: _round(rng.standard_normal((B, T, h, d)), BF) for n, h in (("q", H), ("k", Hk), ("v", Hk), ("g", H))}
    t = {n: _dev(x, BF) for n, x in a.items()}
    # values where a projection left them, behind its queries and keys
    wide = torch.full((B, T, (H + 2 * Hk) * d), float("nan"), dtype=BF, device="cuda")
    wide[..., (H + Hk) * d:] = t["v"].flatten(2)
    t["v"] = wide[..., (H + Hk) * d:].unflatten(2, (Hk, d))
    return a, t, dict(window=W, sinks=S, cu_seqlens=_ints(cu))


@pytest.mark.parametrize("case", WINDOW, ids=lambda c: "-".join(map(str, c[:7])) + ("p" if c[7] else ""))
def test_window_forward(case):
    a, t, kw = _window_inputs(case)
    out, lse = attention.window_attention_fwd(t["q"], t["k"], t["v"], save_for_backward=True, **kw)
    ref, ref_lse = A.window_fwd(a["q"], a["k"], a["v"], case[5], case[6], cu=case[7])
    assert gdn.gdn_get_last_device_error() == 0
    _close(out, ref, TOL_BF16, "out")
    _close(lse, ref_lse, TOL_PAR, "lse")
    assert torch.equal(out, attention.window_attention_fwd(t["q"], t["k"], t["v"], **kw))


@pytest.mark.parametrize("case", WINDOW, ids=lambda c: "-".join(map(str, c[:7])) + ("p" if c[7] else ""))
def test_window_gradients(case):
    a, t, kw = _window_inputs(case)
    out, lse = attention.window_attention_fwd(t["q"], t["k"], t["v"], save_for_backward=True, **kw)
    r = attention.window_attention_bwd(t["q"], t["k"], t["v"], out, lse, t["g"], **kw)
    ref = A.window_bwd(a["q"], a["k"], a["v"], a["g"], case[5], case[6], cu=case[7])
    assert gdn.gdn_get_last_device_error() == 0
    # a token that sees itself alone has no gradient but that of its value; what
    # is left of dP - delta there is the rounding of the output inside delta
    size = np.linalg.norm(ref["dv"])
    for n, want in ref.items():
        if np.linalg.norm(want) <= 1e-2 * size:
            assert np.linalg.norm(_np(r[n]) - want) <= TOL_GRAD * size, n
        else:
            _close(r[n], want, TOL_GRAD, n)
    again = attention.window_attention_bwd(t["q"], t["k"], t["v"], out, lse, t["g"], **kw)
    assert all(torch.equal(r[n], again[n]) for n in r)


STEP = [  # B, H, Hk, d, window, sinks, lengths
    (1, 1, 1, 64, 1, 0, [0]),
    (3, 4, 2, 64, 5, 0, [0, 4, 5]),
    (4, 8, 2, 128, 16, 4, [3, 4, 19, 20]),
    (5, 6, 2, 128, 33, 7, [0, 39, 40, 41, 1000000]),
    (2, 40, 2, 64, 70, 128, [150, 2 ** 31 - 2]),  # twenty heads to a key head
    (2, 16, 1, 128, 1500, 0, [1499, 4000]),       # several blocks to a row
    (1, 5, 5, 64, 4096, 3, [4000]),
]


def _step_inputs(case, seed=0):
    B, H, Hk, d, W, S, lengths = case
    rng = np.random.default_rng(B + H + W + seed)
    a = {n: _round(rng.standard_normal(s), BF) for n, s in
         (("q", (B, H, d)), ("k", (B, Hk, d)), ("v", (B, Hk, d)), ("kc", (B, S + W, Hk, d)), ("vc", (B, S + W, Hk, d)))}
    return a, {n: _dev(x, BF) for n, x in a.items()}, _ints(lengths)


@pytest.mark.parametrize("case", STEP, ids=lambda c: "-".join(map(str, c[:6])))
def test_window_step(case):
    a, t, lengths = _step_inputs(case)
    S = case[5]
    for b, n in enumerate(case[6]):  # rows that hold no token may hold anything
        t["kc"][b, n + 1:], t["vc"][b, n + 1:] = float("nan"), float("inf")
    kc, vc = t["kc"].clone(), t["vc"].clone()
    out = attention.window_attention_step(t["q"], t["k"], t["v"], kc, vc, lengths, sinks=S)
    ref, _, _ = A.window_step(a["q"], a["k"], a["v"], a["kc"], a["vc"], case[6], S)
    assert gdn.gdn_get_last_device_error() == 0
    _close(out, ref, TOL_BF16, "out")
    for b, n in enumerate(case[6]):
        at = A.cache_row(n, case[4], S)
        t["kc"][b, at], t["vc"][b, at] = t["k"][b], t["v"][b]
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))  # noqa: E731  (NaN too)
    assert same(kc, t["kc"]) and same(vc, t["vc"])


def test_window_step_slots_and_idle_rows():
    case = (5, 4, 2, 64, 12, 2, [3, 100, 7, -1, 13])
    a, t, lengths = _step_inputs(case)
    slots = _ints([4, -1, 0, 2, 1])
    kc, vc = t["kc"].clone(), t["vc"].clone()
    out = attention.window_attention_step(t["q"], t["k"], t["v"], kc, vc, lengths, sinks=2, slots=slots)
    ref, kr, vr = A.window_step(a["q"], a["k"], a["v"], a["kc"], a["vc"], case[6], 2, slots=[4, -1, 0, -1, 1])
    _close(out, ref, TOL_BF16, "out")
    assert np.array_equal(_np(kc), kr) and np.array_equal(_np(vc), vr)
    assert out[1].abs().max() == 0 and out[3].abs().max() == 0 and gdn.gdn_get_last_device_error() == 0
    out = attention.window_attention_step(t["q"], t["k"], t["v"], kc, vc, lengths, sinks=2, slots=_ints([4, 5, 0, 2, 1]))
    assert out[1].abs().max() == 0 and gdn.gdn_get_last_device_error() == 7


@pytest.mark.parametrize("cu", [None, [0, 0, 1, 30, 100, 240]])
def test_steps_continue_prompts(cu):
    """A prompt, its cache, and the tokens after it are the longer prompt."""
    H, Hk, d, W, S, more = 4, 2, 64, 40, 3, 6
    B, T = (1, cu[-1]) if cu else (3, 61)
    lens = [T] * B if cu is None else list(np.diff(cu))
    N = len(lens)
    rng = np.random.default_rng(7)
    whole = [{n: _round(rng.standard_normal((1, ln + more, h, d)), BF) for n, h in (("q", H), ("k", Hk), ("v", Hk))}
             for ln in lens]
    prompt = {n: np.concatenate([w[n][:, :ln] for w, ln in zip(whole, lens)], 1 if cu else 0) for n in "qkv"}
    kc, vc = (torch.full((N + 2, S + W, Hk, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    slots = _ints(list(range(N + 1, 1, -1)))
    attention.window_cache_fill(_dev(prompt["k"], BF), _dev(prompt["v"], BF), kc, vc, sinks=S, cu_seqlens=_ints(cu),
                                slots=slots)
    assert torch.isnan(kc[:2]).all()
    want = [A.window_fwd(w["q"], w["k"], w["v"], W, S)[0] for w in whole]
    for s in range(more):
        at = [ln + s for ln in lens]
        row = {n: _dev(np.stack([w[n][0, p] for w, p in zip(whole, at)]), BF) for n in "qkv"}
        out = attention.window_attention_step(row["q"], row["k"], row["v"], kc, vc, _ints(at), sinks=S, slots=slots)
        _close(out, np.stack([w[0, p] for w, p in zip(want, at)]), TOL_BF16, f"step {s}")
    assert gdn.gdn_get_last_device_error() == 0


def test_a_masked_value_has_no_part():
    """NaN and infinities where a token does not look have no part in its output.
    (Rows that share a block with one are computed again with unrounded weights:
    the same to the roundings of the weights, 1.65e-3, that the tolerance has for
    them, and not bit for bit.)"""
    case = (1, 400, 4, 2, 64, 60, 2, [0, 150, 400])
    a, t, kw = _window_inputs(case)
    good = attention.window_attention_fwd(t["q"], t["k"], t["v"], **kw)
    k, v = t["k"].clone(), t["v"].clone()
    for p, x in ((149, float("nan")), (160, float("inf")), (390, float("nan"))):
        k[0, p, 0, 3] = v[0, p, 1, 5] = x
    out = attention.window_attention_fwd(t["q"], k, v, **kw)
    seen = torch.zeros(400, dtype=torch.bool, device="cuda")
    for p, t0, t1 in ((149, 0, 150), (160, 150, 400), (390, 150, 400)):
        seen[p:min(p + 60, t1)] = True
    want = A.window_fwd(a["q"], a["k"], a["v"], 60, 2, cu=case[7])[0]
    _close(out[0, ~seen], want[0, ~seen.cpu().numpy()], TOL_BF16, "rows that do not look there")
    # the first sequence's first tile looks at none of the blocks that hold one
    assert torch.equal(out[0, :128], good[0, :128])
    lo, hi = torch.isfinite(out[0, seen][:, :2]), torch.isfinite(out[0, seen][:, 2:])
    assert not lo.all() and not hi.all()


def test_a_bad_sequence_leaves_the_others_gradients():
    case = (1, 400, 4, 2, 64, 60, 2, [0, 150, 290, 400])
    a, t, kw = _window_inputs(case)
    def both(q, k, v, g):
        out, lse = attention.window_attention_fwd(q, k, v, save_for_backward=True, **kw)
        return attention.window_attention_bwd(q, k, v, out, lse, g, **kw)
    good = both(t["q"], t["k"], t["v"], t["g"])
    bad = {n: t[n].clone() for n in "qkvg"}
    for n in "qkvg":
        bad[n][0, 150:290] = float("nan")
    r = both(bad["q"], bad["k"], bad["v"], bad["g"])
    for n in r:
        assert torch.equal(r[n][0, :150], good[n][0, :150]) and torch.equal(r[n][0, 290:], good[n][0, 290:]), n


def test_large_scores_and_growing_maxima():
    """Scores up to thousands, the largest last: the running maximum moves often."""
    case = (1, 500, 2, 2, 64, 400, 4, None)
    a, t, kw = _window_inputs(case)
    ramp = np.linspace(0.1, 40, 500)[None, :, None, None]
    a["k"] = _round(a["k"] * ramp, BF)
    t["k"] = _dev(a["k"], BF)
    out, lse = attention.window_attention_fwd(t["q"], t["k"], t["v"], save_for_backward=True, **kw)
    ref, ref_lse = A.window_fwd(a["q"], a["k"], a["v"], 400, 4)
    # a score of s has an fp32 error of 2^-22 s (64 products of like size), which is
    # a relative error of its weight: 400 x 2^-22 = 1e-4
    _close(out, ref, TOL_BF16 + 1e-4, "out")
    _close(lse, ref_lse, TOL_PAR, "lse")


def test_window_autograd_and_scale():
    case = (1, 45, 4, 2, 64, 9, 2, [0, 20, 45])
    a, t, kw = _window_inputs(case)
    leaves = [t[n].clone().requires_grad_() for n in "qkv"]
    out = attention.window_attention(*leaves, scale=0.2, **kw)
    (out.float() * t["g"].float()).sum().backward()
    ref = A.window_bwd(a["q"], a["k"], a["v"], a["g"], 9, 2, scale=0.2, cu=[0, 20, 45])
    rng = np.random.default_rng(3)
    for n, leaf in zip("qkv", leaves):
        _close(leaf.grad, ref["d" + n], TOL_GRAD, n)
        # and the definition's own gradient against differences
        way, h = rng.standard_normal(a[n].shape), 1e-5
        ends = [(A.window_fwd(*(a[m] + (s * h * way if m == n else 0) for m in "qkv"), 9, 2, 0.2, [0, 20, 45])[0] * a["g"]).sum()
                for s in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * h)
        assert abs((ref["d" + n] * way).sum() - slope) <= 1e-6 * np.abs(ref["d" + n] * way).sum()
    with torch.no_grad():
        assert torch.equal(attention.window_attention(*leaves, scale=0.2, **kw), out)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        y = attention.window_attention(*leaves, **kw)
        d, = torch.autograd.grad(y.float().sum(), leaves[0], create_graph=True)
        d.float().sum().backward()


def test_window_misaligned_slices_and_streams():
    """Slices that start anywhere, another stream, a captured forward and backward."""
    case = (2, 200, 4, 2, 64, 70, 3, None)
    a, t, kw = _window_inputs(case)
    want, lse = attention.window_attention_fwd(t["q"], t["k"], t["v"], save_for_backward=True, **kw)
    grads = attention.window_attention_bwd(t["q"], t["k"], t["v"], want, lse, t["g"], **kw)
    wide = torch.zeros(2, 200, 3 + 8 * 64, dtype=BF, device="cuda")
    wide[..., 3:3 + 4 * 64], wide[..., 3 + 256:3 + 384], wide[..., 3 + 384:] = (t[n].flatten(2) for n in "qkv")
    q, k, v = (wide[..., 3 + o:3 + o + h * 64].unflatten(2, (h, 64)) for o, h in ((0, 4), (256, 2), (384, 2)))
    assert torch.equal(attention.window_attention_fwd(q, k, v, **kw), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse2 = attention.window_attention_fwd(q, k, v, save_for_backward=True, stream=s, **kw)
    r = attention.window_attention_bwd(q, k, v, out, lse2, t["g"], stream=s, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want) and all(torch.equal(r[n], grads[n]) for n in r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = attention.window_attention_fwd(t["q"], t["k"], t["v"], save_for_backward=True, **kw)
        rg = attention.window_attention_bwd(t["q"], t["k"], t["v"], og, lg, t["g"], **kw)
    for _ in range(2):
        og.zero_()
        graph.replay()
        assert torch.equal(og, want) and all(torch.equal(rg[n], grads[n]) for n in rg)
    assert gdn.gdn_get_last_device_error() == 0


def test_a_score_of_minus_infinity_has_no_weight():
    """A key that a token sees with a score of -inf weighs nothing, also where the
    row is computed again because of a NaN that it does not see."""
    case = (1, 300, 4, 2, 64, 60, 2, None)
    a, t, kw = _window_inputs(case)
    a["q"][..., 3] = np.abs(a["q"][..., 3]) + 0.5
    a["q"] = _round(a["q"], BF)
    a["k"][0, 0, :, 3] = -np.inf
    with np.errstate(invalid="ignore"):
        want, want_lse = A.window_fwd(a["q"], a["k"], a["v"], 60, 2)
    assert np.isfinite(want[0, 1:]).all()
    v = t["v"].clone()
    v[0, 150] = float("nan")
    out, lse = attention.window_attention_fwd(_dev(a["q"], BF), _dev(a["k"], BF), v, save_for_backward=True, **kw)
    rows = np.r_[1:150, 210:300]  # the first token sees that key alone, and 150 to 209 the NaN
    _close(out[0, rows], want[0, rows], TOL_BF16, "out")
    _close(lse[0][:, rows], want_lse[0][:, rows], TOL_PAR, "lse")
    assert torch.isnan(out[0, 0]).all()


@pytest.mark.parametrize("case", [(8, 16, 4, 128, 1024, 4, [1100] * 8), (16, 8, 8, 64, 300, 0, [299] * 16),
                                  (1, 40, 1, 128, 9000, 0, [9500])], ids=lambda c: "-".join(map(str, c[:6])))
def test_a_step_is_off_by_its_outputs_rounding(case):
    """The weights of the second product keep eleven bits or more, so beside the
    rounding of the output there is at most 2^-11 of a weight, in random directions:
    2^-11 / sqrt(3) x 0.72 = 2.1e-4 of L2, which adds in squares (a root mean square
    over 5000 values and more varies by a hundredth or two)."""
    a, t, lengths = _step_inputs(case)
    out = attention.window_attention_step(t["q"], t["k"], t["v"], t["kc"], t["vc"], lengths, sinks=case[5])
    ref, _, _ = A.window_step(a["q"], a["k"], a["v"], a["kc"], a["vc"], case[6], case[5])
    rounding = metrics.rel_l2(_round(ref, BF), ref)
    err = metrics.rel_l2(_np(out), ref)
    assert err ** 2 <= (1.03 * rounding) ** 2 + 2.1e-4 ** 2, (err, rounding)


def test_an_infinite_value_stays_one_in_a_step():
    case = (2, 4, 2, 128, 50, 0, [70, 70])
    a, t, lengths = _step_inputs(case)
    t["vc"][0, 7, 1, 5], t["vc"][1, 9, 0, 100] = float("inf"), float("-inf")
    out = attention.window_attention_step(t["q"], t["k"], t["v"], t["kc"], t["vc"], lengths)
    ref, _, _ = A.window_step(a["q"], a["k"], a["v"], a["kc"], a["vc"], case[6], 0)
    bad = np.zeros(ref.shape, bool)
    bad[0, 2:, 5] = bad[1, :2, 100] = True
    got = _np(out)
    assert np.all(got[0, 2:, 5] == np.inf) and np.all(got[1, :2, 100] == -np.inf)
    _close(np.where(bad, 0, got), np.where(bad, 0, ref), TOL_BF16, "the others")
