"""The mixer operators (short convolution, selective state space scan, group
norm with an activation) against their fp64 definitions.

Tolerances (relative L2 of a tensor), fixed before the first run.
- bf16 outputs carry one rounding (unit roundoff 2^-8, 8 significant bits),
  about 1.65e-3 in L2 over random mantissas; 3e-3 is this package's bound for
  such outputs.  It says nothing of a handful of values: below 16 the bound is
  the rounding itself, 2^-8, and the fp32 bound beside it.
- fp32 outputs of the convolution and the norm are sums of tens of products
  with a few ulp of exp and division: 2e-6 (about 30 x 2^-24).
- fp32 outputs of the scan accumulate an error of at most 2^-22 + 2^-23 |x| per
  decay exp(x) over a memory of up to T steps, in random directions: sqrt(T)
  x 3e-7 is 5e-6 at T = 300; 1e-5.
- fp32 parameter gradients are sums over all rows that may cancel: 3e-5 where
  the terms carry the scan's error, 1e-5 otherwise.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import gdn, mixer  # noqa: E402
from oracle import metrics  # noqa: E402
from oracle import mixer as M  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL_BF16, TOL_F32, TOL_SCAN, TOL_PAR, TOL_SCAN_PAR = 3e-3, 2e-6, 1e-5, 1e-5, 3e-5


def _dev(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda").to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _strided(a, dtype, left=3, right=2):
    """The rows of `a` as a slice of a wider tensor (odd offset and stride)."""
    flat = a.reshape(a.shape[0], a.shape[1], -1) if a.ndim > 2 else a.reshape(a.shape[0], -1)
    wide = np.full(flat.shape[:-1] + (flat.shape[-1] + left + right,), np.nan, np.float32)
    wide[..., left:left + flat.shape[-1]] = flat
    t = _dev(wide, dtype)[..., left:left + flat.shape[-1]]
    return t if a.ndim <= 3 and flat.shape == a.shape else t.unflatten(-1, a.shape[-2:])


def _close(got, want, tol, what):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    if np.abs(want).max(initial=0.0) == 0.0:
        assert np.abs(got).max(initial=0.0) == 0.0, what
        return
    if tol == TOL_BF16 and want.size < 16:
        tol = 2.0 ** -8 + TOL_SCAN
    e = metrics.rel_l2(got, want)
    assert e <= tol, f"{what}: rel L2 {e:.3e} > {tol:.1e}"


def _io_tol(dtype, f32_tol):
    return TOL_BF16 if dtype == BF else f32_tol


def _no_device_error():
    assert gdn.gdn_get_last_device_error() == 0


def _round(a, dtype):
    """What the device holds of a, in fp64."""
    return _np(torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype))


# ----------------------------------------------------------------- convolution

CONV = [  # B, T, D, W, cu, initial state, strided
    (1, 1, 1, 4, None, False, False),
    (2, 0, 8, 4, None, True, False),
    (3, 2, 24, 4, None, True, False),     # shorter than the window
    (2, 77, 64, 4, None, False, False),
    (2, 65, 40, 3, None, True, True),     # rows that no wide access fits
    (1, 130, 129, 2, None, True, False),  # an odd width
    (1, 70, 48, 4, [0, 0, 1, 3, 3, 64, 70], True, False),
    (1, 200, 34, 3, [0, 130, 130, 131, 200], False, True),
    (1, 4096, 520, 4, [0, 17, 2000, 4096], True, False),
]


def _conv_inputs(case, dtype):
    B, T, D, W, cu, state, strided = case
    rng = np.random.default_rng(B + T + D)
    N = len(cu) - 1 if cu else B
    a = dict(x=_round(rng.standard_normal((B, T, D)), dtype), w=_round(rng.uniform(-0.6, 0.6, (D, W)), F32),
             b=_round(rng.uniform(-0.2, 0.2, D), F32), dy=_round(rng.standard_normal((B, T, D)), dtype),
             dfs=_round(rng.standard_normal((N, W - 1, D)), dtype),
             h=_round(rng.standard_normal((N, W - 1, D)), dtype) if state else None)
    t = dict(x=_strided(a["x"], dtype) if strided else _dev(a["x"], dtype), w=_dev(a["w"]), b=_dev(a["b"]),
             dy=_dev(a["dy"], dtype), dfs=_dev(a["dfs"], dtype), h=None if a["h"] is None else _dev(a["h"], dtype),
             cu=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"))
    return a, t


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CONV, ids=str)
def test_conv(case, dtype):
    a, t = _conv_inputs(case, dtype)
    cu = case[4]
    for kind, bias in (("silu", True), ("none", False)):
        b, tb = (a["b"], t["b"]) if bias else (None, None)
        y, fs = mixer.short_conv_fwd(t["x"], t["w"], tb, kind, t["h"], t["cu"], output_final_state=True)
        y_ref, fs_ref = M.conv_fwd(a["x"], a["w"], b, kind, a["h"], cu)
        tol = _io_tol(dtype, TOL_F32)
        _close(y, y_ref, tol, "y")
        assert np.array_equal(_np(fs), fs_ref), "the final state is a copy"
        r = mixer.short_conv_bwd(t["x"], t["w"], t["dy"], tb, kind, t["h"], t["cu"], t["dfs"] if bias else None)
        ref = M.conv_bwd(a["x"], a["w"], a["dy"], b, kind, a["h"], cu, a["dfs"] if bias else None)
        assert ("dbias" in r) == bias and ("d_initial_state" in r) == (a["h"] is not None)
        for k, v in r.items():
            _close(v, ref[k], TOL_PAR if k in ("dweight", "dbias") else tol, k)
    _no_device_error()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,W,strided", [(64, 4, False), (33, 4, False), (48, 2, True)])
def test_conv_steps_continue_a_prompt(dtype, D, W, strided):
    rng = np.random.default_rng(D)
    B, T, more = 3, 21, 5
    x = _round(rng.standard_normal((B, T + more, D)), dtype)
    w, b = _round(rng.uniform(-0.6, 0.6, (D, W)), F32), _round(rng.uniform(-0.2, 0.2, D), F32)
    want, fs_want = M.conv_fwd(x, w, b)
    _, state = mixer.short_conv_fwd(_dev(x[:, :T], dtype), _dev(w), _dev(b), output_final_state=True)
    for t in range(T, T + more):
        xt = _strided(x[:, t], dtype) if strided else _dev(x[:, t], dtype)
        y = mixer.short_conv_step(xt, state, _dev(w), _dev(b))
        _close(y, want[:, t], _io_tol(dtype, TOL_F32), f"step {t}")
    assert np.array_equal(_np(state), fs_want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [2, 70])
def test_conv_of_even_widths(dtype, D):
    """Widths that two channels per thread fit and four do not: the prompt, its
    gradients, and steps through slots."""
    rng = np.random.default_rng(D)
    T, W, S = 45, 4, 6
    x, dy = (_round(rng.standard_normal((2, T, D)), dtype) for _ in range(2))
    w, b = _round(rng.uniform(-0.6, 0.6, (D, W)), F32), _round(rng.uniform(-0.2, 0.2, D), F32)
    want, fs_want = M.conv_fwd(x, w, b)
    grads = M.conv_bwd(x, w, dy, b)
    got = mixer.short_conv_bwd(_dev(x, dtype), _dev(w), _dev(dy, dtype), _dev(b))
    _close(got["dx"], grads["dx"], _io_tol(dtype, TOL_F32), "dx")
    for k in ("dweight", "dbias"):
        _close(got[k], grads[k], TOL_PAR, k)
    cache = torch.zeros(S, W - 1, D, dtype=dtype, device="cuda")
    slots = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    for t in range(T):
        y = mixer.short_conv_step(_dev(x[:, t], dtype), cache, _dev(w), _dev(b), slots=slots)
        _close(y, want[:, t], _io_tol(dtype, TOL_F32), f"step {t}")
    assert np.array_equal(_np(cache)[[4, 1]], fs_want)
    assert not _np(cache)[[0, 2, 3, 5]].any()


# ------------------------------------------------------------------------ scan

SCAN = [  # B, T, D, G, N, cu, initial state, strided, gated, softplus
    (1, 1, 1, 1, 16, None, False, False, True, True),
    (2, 0, 8, 1, 16, None, True, False, True, True),
    (2, 16, 8, 1, 16, None, True, False, True, True),
    (2, 33, 24, 1, 16, None, False, False, True, True),
    (2, 47, 21, 1, 16, None, True, True, True, True),   # odd width, odd strides
    (1, 40, 40, 2, 8, None, True, False, False, True),
    (1, 35, 18, 3, 32, None, True, False, True, False),  # a block that ends inside a group
    (1, 50, 6, 2, 64, None, True, True, True, True),
    (1, 19, 5, 1, 128, None, True, False, True, True),
    (1, 75, 16, 1, 16, [0, 0, 1, 17, 17, 60, 75], True, False, True, True),
    (1, 90, 10, 2, 8, [0, 31, 90], False, True, True, True),
    (1, 300, 4, 1, 16, [0, 299, 300], True, False, False, False),
    (1, 300, 70, 1, 32, None, False, False, True, True),
]


def _scan_inputs(case, dtype):
    B, T, D, G, N, cu, state, strided, gated, soft = case
    rng = np.random.default_rng(T + D + N)
    nseq = len(cu) - 1 if cu else B
    r = lambda v, to=dtype: _round(v, to)  # noqa: E731
    a = dict(u=r(rng.standard_normal((B, T, D)) * 0.7), A=r(-rng.uniform(0.3, 1.5, (D, N)) * np.arange(1, N + 1), F32),
             B=r(rng.standard_normal((B, T, G, N))), C=r(rng.standard_normal((B, T, G, N))),
             D=r(rng.uniform(0.5, 1.5, D), F32), dout=r(rng.standard_normal((B, T, D))),
             dt=r(rng.standard_normal((B, T, D)) if soft else rng.uniform(0.001, 0.3, (B, T, D))),
             z=r(rng.standard_normal((B, T, D))) if gated else None,
             bias=r(rng.uniform(-5, -1, D), F32) if soft else None,
             h=r(rng.standard_normal((nseq, D, N)), F32) if state else None,
             dfs=r(rng.standard_normal((nseq, D, N)), F32))
    act = _strided if strided else _dev
    t = {k: None if v is None else act(v, dtype) if k in ("u", "dt", "z", "B", "C") else
         _dev(v, dtype if k == "dout" else F32) for k, v in a.items()}
    t["cu"] = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    return a, t


def _scan_check(case, dtype):
    a, t = _scan_inputs(case, dtype)
    cu, soft = case[5], case[9]
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["bias"], dt_softplus=soft, initial_state=t["h"], cu_seqlens=t["cu"])
    args = (t["u"], t["dt"], t["A"], t["B"], t["C"])
    o_ref, fs_ref = M.scan_fwd(a["u"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], soft, a["h"], cu)
    out, fs = mixer.ssm_scan_fwd(*args, **kw)
    tol = _io_tol(dtype, TOL_SCAN)
    _close(out, o_ref, tol, "out")
    _close(fs, fs_ref, TOL_SCAN, "final_state")
    out2, fs2, saved = mixer.ssm_scan_fwd(*args, save_for_backward=True, **kw)
    assert torch.equal(out, out2) and torch.equal(fs, fs2)
    for dfs in (None, t["dfs"]):
        r = mixer.ssm_scan_bwd(*args, t["dout"], saved, d_final_state=dfs, **kw)
        ref = M.scan_bwd(a["u"], a["dt"], a["A"], a["B"], a["C"], a["dout"], a["D"], a["z"], a["bias"], soft, a["h"],
                         cu, None if dfs is None else a["dfs"])
        given = {"dz": "z", "ddt_bias": "bias", "d_initial_state": "h"}
        assert set(r) == {k for k in ref if given.get(k) is None or t[given[k]] is not None}
        for k, v in r.items():
            par = k in ("dA", "dD", "ddt_bias")
            _close(v, ref[k], TOL_SCAN_PAR if par else TOL_SCAN if k == "d_initial_state" else tol, k)
        again = mixer.ssm_scan_bwd(*args, t["dout"], saved, d_final_state=dfs, **kw)
        assert all(torch.equal(r[k], again[k]) for k in r), "the same inputs give the same bits"
    _no_device_error()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", SCAN, ids=str)
def test_scan(case, dtype):
    _scan_check(case, dtype)


# Few channels and many tokens: the scan runs in segments joined afterwards.
LONG = [
    (1, 1100, 20, 1, 16, None, True, False, True, True),
    (2, 700, 9, 1, 8, None, False, True, False, True),
    (1, 1500, 18, 2, 32, [0, 700, 700, 701, 1400, 1500], True, False, True, True),
    (1, 640, 3, 1, 64, [0, 1, 640], True, True, True, False),
    (1, 520, 4, 1, 128, None, True, False, True, True),
    (1, 2600, 3, 1, 16, None, True, False, True, True),           # more segments than are joined on the way
    (1, 2700, 5, 1, 8, [0, 2500, 2500, 2700], True, False, True, True),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", LONG, ids=str)
def test_long_scan(case, dtype):
    B, T, D, G, N, cu = case[:6]
    assert gdn.load().gdn_ssm_fwd_workspace_size(len(cu) - 1 if cu else B, T, D, G, N, int(cu is not None)) > 0
    _scan_check(case, dtype)


def test_scan_without_skip_or_bias():
    a, t = _scan_inputs(SCAN[4], F32)
    args = (t["u"], t["dt"], t["A"], t["B"], t["C"])
    out, fs, saved = mixer.ssm_scan_fwd(*args, save_for_backward=True)
    ref, fs_ref = M.scan_fwd(a["u"], a["dt"], a["A"], a["B"], a["C"])
    _close(out, ref, TOL_SCAN, "out")
    _close(fs, fs_ref, TOL_SCAN, "final_state")
    r = mixer.ssm_scan_bwd(*args, t["dout"], saved)
    g = M.scan_bwd(a["u"], a["dt"], a["A"], a["B"], a["C"], a["dout"])
    assert set(r) == {"du", "ddt", "dA", "dB", "dC"}
    for k, v in r.items():
        _close(v, g[k], TOL_SCAN_PAR if k == "dA" else TOL_SCAN, k)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D,G,N,strided", [(24, 1, 16, False), (21, 3, 8, True), (6, 2, 128, False), (10, 1, 64, False)])
def test_scan_steps_continue_a_prompt(dtype, D, G, N, strided):
    T, more = 18, 4
    a, t = _scan_inputs((2, T + more, D, G, N, None, True, False, True, True), dtype)
    o_ref, fs_ref = M.scan_fwd(a["u"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"], a["bias"], True, a["h"])
    cut = {k: t[k][:, :T] for k in ("u", "dt", "z", "B", "C")}
    if D > 6:  # slices of a longer batch are not evenly spaced rows
        with pytest.raises(ValueError, match="evenly spaced"):
            mixer.ssm_scan_fwd(cut["u"], cut["dt"], t["A"], cut["B"], cut["C"])
    cut = {k: v.contiguous() for k, v in cut.items()}
    _, state = mixer.ssm_scan_fwd(cut["u"], cut["dt"], t["A"], cut["B"], cut["C"], t["D"], cut["z"], t["bias"],
                                  initial_state=t["h"])
    for i in range(T, T + more):
        x = {k: _strided(a[k][:, i], dtype) if strided and a[k].ndim == 3 else t[k][:, i].contiguous()
             for k in ("u", "dt", "z", "B", "C")}
        y = mixer.ssm_scan_step(x["u"], x["dt"], t["A"], x["B"], x["C"], state, t["D"], x["z"], t["bias"])
        _close(y, o_ref[:, i], _io_tol(dtype, TOL_SCAN), f"step {i}")
    _close(state, fs_ref, TOL_SCAN, "state")


def test_steps_with_slots():
    """Rows of a cache in any order, idle rows (-1), and a slot outside the
    cache: reported, and nothing is touched."""
    rng = np.random.default_rng(8)
    B, S, D, N, W = 5, 9, 12, 16, 4
    cache = rng.standard_normal((S, D, N))
    conv = rng.standard_normal((S, W - 1, D))
    a, t = _scan_inputs((1, B, D, 1, N, None, False, False, True, True), F32)
    x = {k: t[k][0] for k in ("u", "dt", "z", "B", "C")}
    w = rng.uniform(-0.6, 0.6, (D, W))
    for slots, bad in (([3, -1, 8, 0, 5], False), ([3, -1, S, 0, 5], True)):
        sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
        state, cstate = _dev(cache), _dev(conv)
        y = _np(mixer.ssm_scan_step(x["u"], x["dt"], t["A"], x["B"], x["C"], state, t["D"], x["z"], t["bias"], slots=sl))
        assert gdn.gdn_get_last_device_error() == (7 if bad else 0)
        yc = _np(mixer.short_conv_step(x["u"], cstate, _dev(w), slots=sl))
        assert gdn.gdn_get_last_device_error() == (7 if bad else 0)
        new, cnew = _round(cache, F32), _round(conv, F32)
        for b, s in enumerate(slots):
            if s < 0 or s >= S:
                assert not y[b].any() and not yc[b].any()
                continue
            one = lambda k: a[k][:, b:b + 1]  # noqa: E731
            o, f = M.scan_fwd(one("u"), one("dt"), a["A"], one("B"), one("C"), a["D"], one("z"), a["bias"], True,
                              new[s][None])
            _close(y[b], o[0, 0], TOL_SCAN, "out")
            new[s] = f[0]
            o, f = M.conv_fwd(one("u"), _round(w, F32), None, "silu", cnew[s][None])
            _close(yc[b], o[0, 0], TOL_F32, "y")
            cnew[s] = f[0]
        _close(state, new, TOL_SCAN, "cache")
        assert np.array_equal(_np(cstate), cnew)


def test_out_of_place_steps_leave_the_state():
    a, t = _scan_inputs((1, 4, 8, 1, 16, None, False, False, True, True), F32)
    x = {k: t[k][0] for k in ("u", "dt", "z", "B", "C")}
    state = torch.randn(4, 8, 16, device="cuda")
    before, to = state.clone(), torch.empty_like(state)
    y = mixer.ssm_scan_step(x["u"], x["dt"], t["A"], x["B"], x["C"], state, out_state=to)
    assert torch.equal(state, before)
    y2 = mixer.ssm_scan_step(x["u"], x["dt"], t["A"], x["B"], x["C"], state)
    assert torch.equal(y, y2) and torch.equal(state, to)


def test_packed_equals_separate_sequences():
    """Bit for bit: a sequence's result does not depend on its neighbours."""
    cu = [0, 5, 5, 40, 41, 90]
    a, t = _scan_inputs((1, 90, 24, 1, 16, cu, True, False, True, True), BF)
    kw = dict(D=t["D"], dt_bias=t["bias"])
    out, fs = mixer.ssm_scan_fwd(t["u"], t["dt"], t["A"], t["B"], t["C"], z=t["z"], initial_state=t["h"],
                                 cu_seqlens=t["cu"], **kw)
    w = torch.randn(24, 4, device="cuda")
    y, ys = mixer.short_conv_fwd(t["u"], w, cu_seqlens=t["cu"], output_final_state=True)
    for n, (p, q) in enumerate(zip(cu[:-1], cu[1:])):
        x = {k: t[k][:, p:q] for k in ("u", "dt", "z", "B", "C")}
        o1, f1 = mixer.ssm_scan_fwd(x["u"], x["dt"], t["A"], x["B"], x["C"], z=x["z"], initial_state=t["h"][n:n + 1], **kw)
        assert torch.equal(o1, out[:, p:q]) and torch.equal(f1[0], fs[n])
        y1, s1 = mixer.short_conv_fwd(x["u"], w, output_final_state=True)
        assert torch.equal(y1, y[:, p:q]) and torch.equal(s1[0], ys[n])


def test_malformed_offsets_are_reported():
    for cu in ([0, 9, 4, 20], [0, 9, 18], [1, 9, 20], [0, -3, 20], [0, 30, 20]):
        a, t = _scan_inputs((1, 20, 8, 1, 16, cu, False, False, True, True), F32)
        mixer.short_conv_fwd(t["u"], torch.ones(8, 4, device="cuda"), cu_seqlens=t["cu"], output_final_state=True)
        assert gdn.gdn_get_last_device_error() == 4, cu
        mixer.ssm_scan_fwd(t["u"], t["dt"], t["A"], t["B"], t["C"], cu_seqlens=t["cu"])
        assert gdn.gdn_get_last_device_error() == 4, cu


def test_extreme_steps():
    """Steps so large that every decay is zero forget the past, steps of zero
    keep the state; nothing becomes infinite or NaN on the way."""
    D, N, T = 8, 16, 40
    A = -torch.arange(1, N + 1, device="cuda", dtype=F32).repeat(D, 1)
    u = torch.randn(1, T, D, device="cuda")
    B, C = torch.randn(1, T, 1, N, device="cuda"), torch.randn(1, T, 1, N, device="cuda")
    h = torch.randn(1, D, N, device="cuda")
    dt = torch.full((1, T, D), 500.0, device="cuda")
    out, fs = mixer.ssm_scan_fwd(u, dt, A, B, C, dt_softplus=True, initial_state=h)
    _close(fs, _np(500.0 * u[0, -1, :, None] * B[0, -1])[None], TOL_SCAN, "forgetting")
    out, fs, saved = mixer.ssm_scan_fwd(u, -1000 * torch.ones_like(dt), A, B, C, initial_state=h, save_for_backward=True)
    assert torch.equal(fs, h)
    r = mixer.ssm_scan_bwd(u, -1000 * torch.ones_like(dt), A, B, C, torch.ones_like(u), saved, initial_state=h)
    assert all(torch.isfinite(v).all() for v in r.values()) and not r["ddt"].any()


# ------------------------------------------------------------------------ norm

NORM = [  # rows, C, groups, strided
    (1, 1, 1, False), (0, 64, 1, False), (3, 128, 1, False), (5, 256, 2, False), (9, 2048, 16, False),
    (7, 96, 3, False), (4, 35, 5, False), (6, 130, 1, True), (5, 1000, 1, False), (5, 999, 1, False),
    (3, 4096, 1, False), (2, 8192, 1, False), (3, 2500, 1, True), (2, 8191, 1, False), (700, 64, 4, False),
    (3, 512, 1, False), (33, 1024, 2, True), (4, 500, 1, False), (3, 1998, 2, False), (2, 4098, 1, False), (2, 700, 1, True),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm(case, dtype):
    rows, C, groups, strided = case
    rng = np.random.default_rng(rows + C)
    x, gate, dy = (_round(rng.standard_normal((rows, C)), dtype) for _ in range(3))
    x = _round(x + 0.3, dtype)
    w, b = _round(rng.uniform(0.5, 1.5, C), F32), _round(rng.uniform(-0.5, 0.5, C), F32)
    act = _strided if strided else _dev
    tx, tg, tdy, tw, tb = act(x, dtype), act(gate, dtype), _dev(dy, dtype), _dev(w), _dev(b)
    for gated, first, center, kind, par in ((True, False, False, "silu", "w"), (True, True, False, "silu", "w"),
                                            (False, False, True, "silu", "wb"), (True, False, True, "sigmoid", "wb"),
                                            (False, False, False, "none", ""), (True, True, True, "silu", "b")):
        if center and C == groups:
            continue  # one value per group: it minus its mean is zero whatever comes in
        pw, pb, g = (w if "w" in par else None), (b if "b" in par else None), (gate if gated else None)
        kw = dict(groups=groups, center=center, gate_first=first)
        targs = dict(weight=None if pw is None else tw, bias=None if pb is None else tb, gate=tg if gated else None,
                     activation=kind, **kw)
        y = mixer.group_norm_fwd(tx, **targs)
        what = (gated, first, center, kind, par)
        _close(y, M.norm_fwd(x, pw, pb, g, kind=kind, **kw), _io_tol(dtype, TOL_F32), what)
        r = mixer.group_norm_bwd(tx, tdy, **targs)
        ref = M.norm_bwd(x, dy, pw, pb, g, kind=kind, **kw)
        for k, v in r.items():
            # with one value per group dx is the difference of equal numbers: only its scale against dy is bounded
            if C == groups and k in ("dx", "dgate"):
                assert np.abs(_np(v) - ref[k]).max(initial=0.0) <= 1e-2 * np.abs(dy).max(initial=0.0), what
                continue
            _close(v, ref[k], TOL_PAR if k in ("dweight", "dbias") else _io_tol(dtype, TOL_F32), (what, k))


def test_norm_of_a_zero_row_and_of_large_values():
    x = torch.zeros(2, 64, device="cuda")
    x[1] = 1e15
    y = mixer.group_norm_fwd(x, activation="none")
    assert not y[0].any()
    _close(y[1], np.ones(64), TOL_F32, "large values")
    r = mixer.group_norm_bwd(x, torch.randn_like(x), activation="none")
    assert torch.isfinite(r["dx"]).all()


def test_norm_takes_any_leading_shape():
    x = torch.randn(2, 3, 4, 128, device="cuda")
    y = mixer.group_norm_fwd(x, gate=x)
    assert torch.equal(y.view(-1, 128), mixer.group_norm_fwd(x.view(-1, 128), gate=x.view(-1, 128)))


# -------------------------------------------------------------------- autograd

def test_autograd_matches_the_explicit_route():
    a, t = _scan_inputs((2, 33, 24, 1, 16, None, True, False, True, True), F32)
    names = ("u", "dt", "A", "B", "C", "D", "z", "bias", "h")
    leaf = {k: t[k].clone().requires_grad_() for k in names}
    out, fs = mixer.ssm_scan(leaf["u"], leaf["dt"], leaf["A"], leaf["B"], leaf["C"], leaf["D"], leaf["z"],
                             leaf["bias"], initial_state=leaf["h"])
    ((out * t["dout"]).sum() + (fs * t["dfs"]).sum()).backward()
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["bias"], initial_state=t["h"])
    args = (t["u"], t["dt"], t["A"], t["B"], t["C"])
    _, _, saved = mixer.ssm_scan_fwd(*args, save_for_backward=True, **kw)
    r = mixer.ssm_scan_bwd(*args, t["dout"], saved, d_final_state=t["dfs"], **kw)
    for k, g in zip(names, ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "d_initial_state")):
        assert torch.equal(leaf[k].grad, r[g]), k
    x = t["u"].clone().requires_grad_()
    w = torch.randn(24, 4, device="cuda", requires_grad=True)
    y, s = mixer.short_conv(x, w)
    n = mixer.group_norm(y, gate=t["z"])
    n.backward(t["dout"])
    dy = mixer.group_norm_bwd(y.detach(), t["dout"], gate=t["z"])["dx"]
    g = mixer.short_conv_bwd(t["u"], w.detach(), dy)
    assert torch.equal(x.grad, g["dx"]) and torch.equal(w.grad, g["dweight"])


def test_gradients_against_differences():
    """Directional differences of the fp32 kernels themselves: the scan's
    rounding over the difference of 2e-2 leaves about 1e-3."""
    a, t = _scan_inputs((1, 20, 16, 1, 16, None, True, False, True, True), F32)
    leaf = {k: t[k].clone().requires_grad_() for k in ("u", "dt", "A", "B", "C", "D", "z", "bias", "h")}

    def f(v):
        out, fs = mixer.ssm_scan(v["u"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["z"], v["bias"],
                                 initial_state=v["h"])
        return (out.double() * t["dout"]).sum() + (fs.double() * t["dfs"]).sum()

    f(leaf).backward()
    gen = torch.Generator(device="cuda").manual_seed(1)
    for k in leaf:
        d = torch.randn(leaf[k].shape, generator=gen, device="cuda")
        d = d / d.norm()
        with torch.no_grad():
            up, down = ({**leaf, k: leaf[k] + s * 1e-2 * d} for s in (1, -1))
            num = float((f(up) - f(down)) / 2e-2)
        got = float((leaf[k].grad.double() * d).sum())
        assert abs(got - num) <= 5e-3 * max(1.0, float(leaf[k].grad.norm())), (k, got, num)


def test_on_another_stream():
    a, t = _scan_inputs((2, 33, 24, 1, 16, None, True, False, True, True), F32)
    args = (t["u"], t["dt"], t["A"], t["B"], t["C"])
    out, fs = mixer.ssm_scan_fwd(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, f2 = mixer.ssm_scan_fwd(*args)
    torch.cuda.current_stream().wait_stream(s)
    o3, f3 = mixer.ssm_scan_fwd(*args, stream=s)
    s.synchronize()
    assert torch.equal(out, o2) and torch.equal(fs, f2) and torch.equal(out, o3) and torch.equal(fs, f3)


@pytest.mark.parametrize("as_address", [False, True])
def test_memory_of_another_stream(monkeypatch, as_address):
    """stream= takes outputs and workspaces from that stream's memory: what the
    current stream gives back or takes meanwhile is not theirs."""
    a, t = _scan_inputs((1, 700, 24, 1, 16, None, True, False, True, True), F32)
    args = (t["u"], t["dt"], t["A"], t["B"], t["C"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    at = []
    plain = mixer._workspace

    def workspace(nbytes, device):
        at.append((nbytes, torch.cuda.current_stream().cuda_stream))
        return plain(nbytes, device)

    monkeypatch.setattr(mixer, "_workspace", workspace)
    stream = s.cuda_stream if as_address else s
    out, fs, saved = mixer.ssm_scan_fwd(*args, save_for_backward=True, stream=stream)
    grads = mixer.ssm_scan_bwd(*args, out, saved, stream=stream)
    s.synchronize()
    assert len(at) == 2 and all(n > 0 and where == s.cuda_stream for n, where in at)
    owner = [(g["address"], g["address"] + g["total_size"], g["stream"]) for g in torch.cuda.memory_snapshot()]
    for x in (out, fs, saved, *grads.values()):
        assert [o for lo, hi, o in owner if lo <= x.data_ptr() < hi] == [s.cuda_stream]


# -------------------------------------------------------------- large offsets

def test_offsets_beyond_32_bits():
    """Rows far apart in a wide tensor and a slot far into a cache: the last
    rows lie beyond 2^32 elements, and equal those of compact inputs."""
    T, D, N, wide = 65600, 64, 16, 65664
    assert (T - 1) * wide > 2 ** 32
    big = torch.empty(1, T, wide, dtype=BF, device="cuda")
    u = torch.randn(1, T, D, device="cuda").to(BF)
    proj = torch.randn(1, T, 2 * N, device="cuda").to(BF)
    big[..., 64:64 + D] = u
    big[..., 256:256 + 2 * N] = proj
    far = big[..., 64:64 + D]
    B, C = (big[..., 256 + i * N:256 + (i + 1) * N].unflatten(2, (1, N)) for i in range(2))
    B1, C1 = (proj[..., i * N:(i + 1) * N].unflatten(2, (1, N)) for i in range(2))
    w = torch.randn(D, 4, device="cuda")
    y, fs = mixer.short_conv_fwd(far, w, output_final_state=True)
    y1, fs1 = mixer.short_conv_fwd(u, w, output_final_state=True)
    assert torch.equal(y, y1) and torch.equal(fs, fs1)
    g, g1 = mixer.short_conv_bwd(far, w, y), mixer.short_conv_bwd(u, w, y)
    assert all(torch.equal(g[k], g1[k]) for k in g)
    A = -torch.rand(D, N, device="cuda")
    o, h = mixer.ssm_scan_fwd(far, far, A, B, C, z=far)
    o1, h1 = mixer.ssm_scan_fwd(u, u, A, B1, C1, z=u)
    assert torch.equal(o, o1) and torch.equal(h, h1)
    n, n1 = mixer.group_norm_fwd(far, gate=far, groups=2), mixer.group_norm_fwd(u, gate=u, groups=2)
    assert torch.equal(n, n1)
    del big, far, B, C
    S, D, N = 16500, 2048, 128
    cache = torch.empty(S, D, N, device="cuda")
    assert (S - 1) * D * N > 2 ** 32
    row = torch.randn(1, D, N, device="cuda")
    cache[S - 1] = row[0]
    x = torch.randn(1, D, device="cuda")
    Bm, A = torch.randn(1, 1, N, device="cuda"), -torch.rand(D, N, device="cuda")
    slot = torch.tensor([S - 1], dtype=torch.int32, device="cuda")
    y = mixer.ssm_scan_step(x, x, A, Bm, Bm, cache, slots=slot)
    y1 = mixer.ssm_scan_step(x, x, A, Bm, Bm, row)
    assert torch.equal(y, y1) and torch.equal(cache[S - 1], row[0])
    _no_device_error()


def test_nan_and_infinity_stay_in_their_sequence():
    """A NaN input of one packed sequence, and infinities in the padding columns
    beside the rows, touch no other sequence."""
    cu = [0, 40, 41, 100]
    a, t = _scan_inputs((1, 100, 24, 1, 16, cu, True, False, True, True), F32)
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["bias"], initial_state=t["h"], cu_seqlens=t["cu"])
    args = (t["dt"], t["A"], t["B"], t["C"])
    out, fs, saved = mixer.ssm_scan_fwd(t["u"], *args, save_for_backward=True, **kw)
    g = mixer.ssm_scan_bwd(t["u"], *args, t["dout"], saved, **kw)
    w = torch.randn(24, 4, device="cuda")
    y, _ = mixer.short_conv_fwd(t["u"], w, cu_seqlens=t["cu"])
    gy = mixer.short_conv_bwd(t["u"], w, t["dout"], cu_seqlens=t["cu"])
    u = t["u"].clone()
    u[0, 40] = float("nan")
    out2, fs2, saved2 = mixer.ssm_scan_fwd(u, *args, save_for_backward=True, **kw)
    g2 = mixer.ssm_scan_bwd(u, *args, t["dout"], saved2, **kw)
    y2, _ = mixer.short_conv_fwd(u, w, cu_seqlens=t["cu"])
    gy2 = mixer.short_conv_bwd(u, w, t["dout"], cu_seqlens=t["cu"])
    assert torch.isnan(out2[0, 40]).all() and torch.isnan(y2[0, 40]).all()
    for rows in (slice(0, 40), slice(41, 100)):
        for p, q in ((out, out2), (y, y2), (gy["dx"], gy2["dx"])) + tuple((g[k], g2[k]) for k in ("du", "ddt", "dz", "dB", "dC")):
            assert torch.equal(p[0, rows], q[0, rows])
    assert torch.equal(fs[0], fs2[0]) and torch.equal(fs[2], fs2[2]) and torch.isnan(fs2[1]).all()
