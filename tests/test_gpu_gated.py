"""The gated linear recurrence against its fp64 definition.

Tolerances (relative L2 of a tensor), fixed before the first run.
- bf16 outputs carry one rounding: 3e-3, this package's bound for them, and the
  rounding itself (2^-8) below 16 values.
- fp32 states: a decay has a relative error of at most 2^-22 + 2^-22 |L|, an
  input gate some 2^-20 (its root halves the error of 1 - a^2, at most 2^-20.4
  where it comes from the exponential), in random directions over a memory of at
  most T steps: sqrt(300) x 3e-7 + 1e-6 < 1e-5.
- gradients of lam are sums over all rows that may cancel: 3e-5.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import gdn, mixer  # noqa: E402
from oracle import metrics  # noqa: E402
from oracle import mixer as M  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL_BF16, TOL_F32, TOL_PAR = 3e-3, 1e-5, 3e-5

CASES = [  # B, T, D, cu, initial state, strided gates
    (1, 1, 1, None, False, False),
    (2, 0, 8, None, True, False),
    (3, 7, 24, None, True, False),             # less than a strip
    (2, 65, 64, None, False, True),            # one block of strips and one token
    (1, 300, 129, None, True, False),          # an odd width
    (2, 1030, 70, None, True, True),           # several rounds of a cluster
    (1, 70, 48, [0, 0, 1, 3, 3, 64, 70], True, False),
    (1, 200, 34, [0, 130, 130, 131, 200], False, True),
    (1, 24, 66, [0, 8, 16, 24], True, False),  # ends on strips
    (1, 9, 5, list(range(10)), True, False),   # a token each
    (1, 4099, 130, [0, 17, 2000, 4096, 4099], True, False),
]


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


def _inputs(case, dtype, seed=0, lam=(-6.0, -2.0)):
    B, T, D, cu, state, strided = case
    rng = np.random.default_rng(B + T + D + seed)
    N = len(cu) - 1 if cu else B
    a = {k: _round(rng.standard_normal((B, T, D)), dtype) for k in ("x", "r", "i", "dy")}
    a["lam"] = _round(rng.uniform(*lam, D), F32)
    a["dfs"] = _round(rng.standard_normal((N, D)), F32)
    a["h0"] = _round(rng.standard_normal((N, D)), F32) if state else None
    t = {k: None if v is None else _dev(v, dtype if k in "x r i dy".split() else F32) for k, v in a.items()}
    if strided:  # both gates in one projection, behind an odd number of other channels
        wide = torch.full((B, T, 3 + 2 * D), float("nan"), dtype=dtype, device="cuda")
        wide[..., 3:3 + D], wide[..., 3 + D:] = t["r"], t["i"]
        t["r"], t["i"] = wide[..., 3:3 + D], wide[..., 3 + D:]
    t["cu"] = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    return a, t


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:3])) + ("p" if c[3] else ""))
def test_forward_and_gradients(case, dtype):
    a, t = _inputs(case, dtype)
    cu = case[3]
    io = TOL_BF16 if dtype == BF else TOL_F32
    kw = dict(initial_state=t["h0"], cu_seqlens=t["cu"])
    y, fs, saved = mixer.gated_scan_fwd(t["x"], t["r"], t["i"], t["lam"], save_for_backward=True, **kw)
    y_ref, fs_ref = M.gated_fwd(a["x"], a["r"], a["i"], a["lam"], h0=a["h0"], cu=cu)
    _close(y, y_ref, io, "y")
    _close(fs, fs_ref, TOL_F32, "final state")
    plain, none = mixer.gated_scan_fwd(t["x"], t["r"], t["i"], t["lam"], output_final_state=False, **kw)
    assert none is None and torch.equal(plain, y)
    for dfs in (None, "dfs"):
        g = mixer.gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], t["dy"], saved,
                                 d_final_state=t["dfs"] if dfs else None, **kw)
        ref = M.gated_bwd(a["x"], a["r"], a["i"], a["lam"], a["dy"], h0=a["h0"], cu=cu, dfs=a["dfs"] if dfs else None)
        assert set(g) == set(ref)
        for k, v in g.items():
            _close(v, ref[k], {"dlam": TOL_PAR, "d_initial_state": TOL_F32}.get(k, io), k)
    assert gdn.gdn_get_last_device_error() == 0


@pytest.mark.parametrize("n", [510, 511, 512, 513, 900])
def test_more_sequences_than_a_block_holds_offsets_of(n):
    """Offsets in shared and in global memory, empty sequences at both ends and between."""
    rng = np.random.default_rng(n)
    lengths = rng.integers(0, 4, n)
    lengths[[0, n // 2, n - 1]] = 0
    lengths[[n // 3, n - 2]] = 90, 300
    cu = np.concatenate([[0], np.cumsum(lengths)]).tolist()
    case = (1, cu[-1], 36, cu, True, False)
    a, t = _inputs(case, F32)
    kw = dict(initial_state=t["h0"], cu_seqlens=t["cu"])
    y, fs, saved = mixer.gated_scan_fwd(t["x"], t["r"], t["i"], t["lam"], save_for_backward=True, **kw)
    y_ref, fs_ref = M.gated_fwd(a["x"], a["r"], a["i"], a["lam"], h0=a["h0"], cu=cu)
    _close(y, y_ref, TOL_F32, "y")
    _close(fs, fs_ref, TOL_F32, "final state")
    g = mixer.gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], t["dy"], saved, d_final_state=t["dfs"], **kw)
    ref = M.gated_bwd(a["x"], a["r"], a["i"], a["lam"], a["dy"], h0=a["h0"], cu=cu, dfs=a["dfs"])
    for k, v in g.items():
        _close(v, ref[k], {"dlam": TOL_PAR}.get(k, TOL_F32), k)
    assert gdn.gdn_get_last_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,strided", [(64, False), (33, False), (48, True)])
def test_steps_continue_a_prompt(dtype, D, strided):
    B, T, more = 3, 21, 5
    a, t = _inputs((B, T + more, D, None, False, strided), dtype)
    y_ref, fs_ref = M.gated_fwd(a["x"], a["r"], a["i"], a["lam"])
    _, state = mixer.gated_scan_fwd(*(t[k][:, :T].contiguous() for k in "xri"), t["lam"])
    for s in range(T, T + more):
        y = mixer.gated_scan_step(t["x"][:, s], t["r"][:, s], t["i"][:, s], t["lam"], state)
        _close(y, y_ref[:, s], TOL_BF16 if dtype == BF else TOL_F32, f"step {s}")
    _close(state, fs_ref, TOL_F32, "state")


def test_step_slots():
    """Idle rows, rows of the cache nobody names, a slot outside the cache."""
    B, S, D = 5, 7, 40
    a, t = _inputs((1, B, D, None, False, False), F32)
    cache = torch.randn(S, D, device="cuda")
    keep = cache.clone()
    slots = torch.tensor([6, -1, 0, 3, -7], dtype=torch.int32, device="cuda")
    row = [t[k][0] for k in "xri"]
    y = mixer.gated_scan_step(*row, t["lam"], cache, slots=slots)
    for b, s in enumerate(slots.tolist()):
        if s < 0:
            assert y[b].abs().max() == 0
            continue
        ref, _ = M.gated_fwd(*(a[k][:, b:b + 1] for k in "xri"), a["lam"], h0=_np(keep[s:s + 1]))
        _close(y[b], ref[0, 0], TOL_F32, f"row {b}")
        assert torch.equal(cache[s], y[b])
    for s in (1, 2, 4, 5):
        assert torch.equal(cache[s], keep[s])
    assert gdn.gdn_get_last_device_error() == 0
    out = torch.zeros_like(cache)
    y2 = mixer.gated_scan_step(*row, t["lam"], keep, slots=slots, out_state=out)
    assert torch.equal(y2, y) and torch.equal(out[6], cache[6]) and out[1].abs().max() == 0
    slots[1] = S
    y3 = mixer.gated_scan_step(*row, t["lam"], keep.clone(), slots=slots)
    assert y3[1].abs().max() == 0 and gdn.gdn_get_last_device_error() == 7


@pytest.mark.parametrize("lam,what", [((-40.0, -20.0), "decays that round to 1"), ((3.0, 30.0), "decays near 0")])
def test_extreme_decays(lam, what):
    """lam far down: L is tiny and 1 - a^2 comes from it, not from a rounded a; far
    up: the memory is gone.  Gates from closed to open."""
    a, t = _inputs((2, 130, 64, None, True, False), F32, lam=lam)
    a["r"][:, ::3] *= 30
    t["r"] = _dev(a["r"])
    a["r"] = _np(t["r"])
    y, fs, saved = mixer.gated_scan_fwd(t["x"], t["r"], t["i"], t["lam"], initial_state=t["h0"], save_for_backward=True)
    y_ref, fs_ref = M.gated_fwd(a["x"], a["r"], a["i"], a["lam"], h0=a["h0"])
    _close(y, y_ref, TOL_F32, what)
    g = mixer.gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], t["dy"], saved, initial_state=t["h0"])
    ref = M.gated_bwd(a["x"], a["r"], a["i"], a["lam"], a["dy"], h0=a["h0"])
    for k, v in g.items():
        _close(v, ref[k], TOL_PAR if k == "dlam" else TOL_F32, k)


@pytest.mark.parametrize("T,cu", [(70, [0, 20, 20, 37, 70]), (2000, [0, 700, 1201, 2000])])
def test_a_nan_stays_in_its_sequence(T, cu):
    a, t = _inputs((1, T, 66, cu, True, False), F32)
    x = t["x"].clone()
    bad = next(n for n in range(1, len(cu) - 1) if cu[n + 1] > cu[n])
    x[0, cu[bad] + 2, :33] = float("nan")
    x[0, cu[bad] + 3, 33:] = float("inf")
    kw = dict(initial_state=t["h0"], cu_seqlens=t["cu"])
    good = mixer.gated_scan_fwd(t["x"], t["r"], t["i"], t["lam"], save_for_backward=True, **kw)
    y, fs, saved = mixer.gated_scan_fwd(x, t["r"], t["i"], t["lam"], save_for_backward=True, **kw)
    g0 = mixer.gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], t["dy"], good[2], **kw)
    g = mixer.gated_scan_bwd(x, t["r"], t["i"], t["lam"], t["dy"], saved, **kw)
    for n in range(len(cu) - 1):
        rows = slice(cu[n], cu[n + 1])
        if n == bad:
            assert not torch.isfinite(y[0, rows]).all()
            continue
        assert torch.equal(y[0, rows], good[0][0, rows]) and torch.equal(fs[n], good[1][n])
        for k in ("dx", "dr", "di"):
            assert torch.equal(g[k][0, rows], g0[k][0, rows]), k
        assert torch.equal(g["d_initial_state"][n], g0["d_initial_state"][n])


def test_autograd_against_differences():
    a, t = _inputs((1, 37, 6, [0, 0, 11, 37], True, False), F32, seed=5)
    leaves = {k: t[k].clone().requires_grad_() for k in ("x", "r", "i", "lam", "h0")}
    y, fs = mixer.gated_scan(leaves["x"], leaves["r"], leaves["i"], leaves["lam"], initial_state=leaves["h0"],
                             cu_seqlens=t["cu"])
    (y * t["dy"]).sum().add((fs * t["dfs"]).sum()).backward()
    rng = np.random.default_rng(1)

    def value(**shift):
        b = {k: a[k] + shift.get(k, 0) for k in leaves}
        yy, ff = M.gated_fwd(b["x"], b["r"], b["i"], b["lam"], h0=b["h0"], cu=[0, 0, 11, 37])
        return (yy * a["dy"]).sum() + (ff * a["dfs"]).sum()

    for k, leaf in leaves.items():
        way, h = rng.standard_normal(a[k].shape), 1e-5
        slope = (value(**{k: h * way}) - value(**{k: -h * way})) / (2 * h)
        # central differences in fp64: h^2 of the third derivative, below 1e-8 of the slope's own size
        got = float((_np(leaf.grad) * way).sum())
        size = float(np.abs(_np(leaf.grad) * way).sum())
        assert abs(got - slope) <= 1e-5 * size + 1e-7 * abs(slope), k


def test_runs_on_a_graph_and_another_stream():
    a, t = _inputs((2, 500, 64, None, True, False), BF)
    args = [t[k] for k in "xri"]
    want, fs_want = mixer.gated_scan_fwd(*args, t["lam"], initial_state=t["h0"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, fs = mixer.gated_scan_fwd(*args, t["lam"], initial_state=t["h0"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want) and torch.equal(fs, fs_want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, fg, saved = mixer.gated_scan_fwd(*args, t["lam"], initial_state=t["h0"], save_for_backward=True)
        g = mixer.gated_scan_bwd(*args, t["lam"], t["dy"], saved, initial_state=t["h0"])
    graph.replay()
    first = {k: v.clone() for k, v in g.items()}
    assert torch.equal(yg, want) and torch.equal(fg, fs_want)
    t["x"].copy_(t["x"].flip(1))
    graph.replay()
    assert not torch.equal(yg, want)
    t["x"].copy_(t["x"].flip(1))
    graph.replay()
    assert torch.equal(yg, want) and all(torch.equal(g[k], first[k]) for k in g)


# Strong decays, channel by channel: a relative L2 norm over a tensor is ruled by the
# weak ones in it.  Per channel of decay L, by the roundings of an fp32 path: softplus
# 2^-22, the gate's sigmoid 2^-21 (an exponential, a sum, a reciprocal), two products
# 2^-23 and the change of base 1.5 x 2^-24, so L is off by 9.3e-7 of itself and a =
# exp(L) by 9.3e-7 |L| + 2^-22.  dr, dlam and d_initial_state are products of a with
# at most eight more factors and sums of some 2^-22 each, and L once more: 4e-6.
DECAYS = np.array([-0.45, -0.52, -0.7, -1.0, -2.0, -4.0, -6.0, -8.0, -10.0, -12.0, -14.0, -16.0, -17.0, -18.0, -25.0, -40.0])


def _tol_of(L):
    return 4e-6 + 1e-6 * np.abs(L)


def _decaying(B, T, seed):
    """Gates about 1/2 and lam by channel, so that its L is about DECAYS."""
    rng = np.random.default_rng(seed)
    D = len(DECAYS)
    lam = _round(np.log(np.expm1(-DECAYS / 4)), F32)
    a = {k: _round(rng.standard_normal((B, T, D)), F32) for k in ("x", "i", "dy")}
    a["r"] = _round(rng.uniform(-0.05, 0.05, (B, T, D)), F32)
    a["h0"] = _round(rng.standard_normal((B, D)), F32)
    gate = 1 / (1 + np.exp(-a["r"]))
    return a, lam, -8 * np.log1p(np.exp(lam)) * gate, gate


@pytest.mark.parametrize("T", [1, 3, 40, 700])
def test_gradients_through_strong_decays(T):
    a, lam, L, gate = _decaying(24, T, T)
    t = {k: _dev(v) for k, v in a.items()}
    args = (t["x"], t["r"], t["i"], _dev(lam))
    _, _, saved = mixer.gated_scan_fwd(*args, initial_state=t["h0"], save_for_backward=True)
    g = mixer.gated_scan_bwd(*args, t["dy"], saved, initial_state=t["h0"])
    ref = M.gated_bwd(a["x"], a["r"], a["i"], lam, a["dy"], h0=a["h0"])
    tol = _tol_of(np.abs(L).max((0, 1)))
    for k, axes in (("dr", (0, 1)), ("d_initial_state", 0)):
        err = np.sqrt(((_np(g[k]) - ref[k]) ** 2).sum(axes) / (ref[k] ** 2).sum(axes))
        assert np.all(err <= tol), (k, err)
    # dlam sums over the rows and may cancel: against the sum of its terms' sizes
    size = (np.abs(ref["dr"] / (L * (1 - gate))) * gate).sum((0, 1)) * 8 / (1 + np.exp(-lam))
    err = np.abs(_np(g["dlam"]) - ref["dlam"]) / size
    assert np.all(err <= tol), err


def test_a_state_through_strong_decays():
    """One token without input: what is left of the state, value by value."""
    a, lam, L, _ = _decaying(24, 1, 3)
    t = {k: _dev(v) for k, v in a.items()}
    want, tol = np.exp(L[:, 0]) * a["h0"], _tol_of(L[:, 0])
    zero = torch.zeros_like(t["x"])
    y, fs = mixer.gated_scan_fwd(zero, t["r"], t["i"], _dev(lam), initial_state=t["h0"])
    step = mixer.gated_scan_step(zero[:, 0], t["r"][:, 0], t["i"][:, 0], _dev(lam), t["h0"].clone())
    for got in (y[:, 0], fs, step):
        assert np.all(np.abs(_np(got) - want) <= tol * np.abs(want))
