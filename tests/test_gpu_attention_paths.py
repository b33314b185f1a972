"""The gated recurrence and the attention operators at the sizes where their
kernels' loops turn, at offsets beyond 32 bits, and in calls that share a GPU.
Tolerances as in test_gpu_attention.py and test_gpu_gated.py."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import attention, gdn, mixer  # noqa: E402
from oracle import attention as A  # noqa: E402
from oracle import metrics  # noqa: E402
from oracle import mixer as M  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL_BF16, TOL_GRAD, TOL_F32, TOL_PAR = 3e-3, 5e-3, 1e-5, 3e-5


def _dev(a, dtype=F32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to("cuda").to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _round(a, dtype):
    return _np(torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype))


def _close(got, want, tol, what):
    got = _np(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape and np.all(np.isfinite(got)), what
    e = metrics.rel_l2(got, want)
    assert e <= tol, f"{what}: rel L2 {e:.3e} > {tol:.1e}"


def _ints(a):
    return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


# tokens around whole tiles (128), windows around them, first tokens around the
# widths of their block (32, 64, 96, 128), stretches that end anywhere
EDGES = [(T, W, S) for T, W, S in (
    (128, 127, 1), (128, 128, 128), (129, 1, 32), (255, 128, 33), (256, 129, 64), (256, 2, 128), (257, 256, 65), (383, 127, 96),
    (384, 255, 97), (385, 128, 31), (640, 1, 128), (641, 130, 127), (1025, 384, 5), (1153, 64, 40))]


@pytest.mark.parametrize("heads", [(2, 1, 64), (3, 1, 128), (2, 2, 128)], ids=str)
@pytest.mark.parametrize("T,W,S", EDGES)
def test_window_edges(T, W, S, heads):
    H, Hk, d = heads
    rng = np.random.default_rng(T + W + S + H)
    a = {n: _round(rng.standard_normal((1, T, h, d)), BF) for n, h in (("q", H), ("k", Hk), ("v", Hk), ("g", H))}
    t = {n: _dev(x, BF) for n, x in a.items()}
    out, lse = attention.window_attention_fwd(t["q"], t["k"], t["v"], W, S, save_for_backward=True)
    ref, ref_lse = A.window_fwd(a["q"], a["k"], a["v"], W, S)
    _close(out, ref, TOL_BF16, "out")
    _close(lse, ref_lse, 1e-5, "lse")
    r = attention.window_attention_bwd(t["q"], t["k"], t["v"], out, lse, t["g"], W, S)
    for n, want in A.window_bwd(a["q"], a["k"], a["v"], a["g"], W, S).items():
        _close(r[n], want, TOL_GRAD, n)
    assert gdn.gdn_get_last_device_error() == 0


@pytest.mark.parametrize("n,most", [(40, 9), (300, 3), (7, 300)])
def test_many_ragged_sequences(n, most):
    """Sequences of any length, empty ones among them, of every operator that packs them."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, most + 1, n)
    cu = [0, *np.cumsum(lens).tolist()]
    T, D = cu[-1], 40
    a = {k: _round(rng.standard_normal((1, T, D)), F32) for k in ("x", "r", "i", "g")}
    lam, h0 = _round(rng.uniform(-5, -2, D), F32), _round(rng.standard_normal((n, D)), F32)
    dfs = _round(rng.standard_normal((n, D)), F32)
    t = {k: _dev(v) for k, v in a.items()}
    kw = dict(initial_state=_dev(h0), cu_seqlens=_ints(cu))
    y, fs, saved = mixer.gated_scan_fwd(t["x"], t["r"], t["i"], _dev(lam), save_for_backward=True, **kw)
    ry, rfs = M.gated_fwd(a["x"], a["r"], a["i"], lam, h0=h0, cu=cu)
    _close(y, ry, TOL_F32, "y")
    _close(fs, rfs, TOL_F32, "final state")
    g = mixer.gated_scan_bwd(t["x"], t["r"], t["i"], _dev(lam), t["g"], saved, d_final_state=_dev(dfs), **kw)
    for k, v in M.gated_bwd(a["x"], a["r"], a["i"], lam, a["g"], h0=h0, cu=cu, dfs=dfs).items():
        _close(g[k], v, TOL_PAR if k == "dlam" else TOL_F32, k)
    q, k, v, go = (_round(rng.standard_normal((1, T, h, 64)), BF) for h in (2, 1, 1, 2))
    f = np.float32(10000.0) ** (-np.arange(32, dtype=np.float32) / 32)
    tq, tk = attention.qk_norm_rope_fwd(_dev(q, BF), _dev(k, BF), inv_freq=_dev(f), cu_seqlens=_ints(cu))
    _close(tq, A.rope_fwd(q, None, f, A.positions_of(q, cu)), TOL_BF16, "rotated q")
    q, k = _np(tq), _np(tk)
    out, lse = attention.window_attention_fwd(tq, tk, _dev(v, BF), 5, 2, cu_seqlens=_ints(cu), save_for_backward=True)
    _close(out, A.window_fwd(q, k, v, 5, 2, cu=cu)[0], TOL_BF16, "attention")
    r = attention.window_attention_bwd(tq, tk, _dev(v, BF), out, lse, _dev(go, BF), 5, 2, cu_seqlens=_ints(cu))
    for name, want in A.window_bwd(q, k, v, go, 5, 2, cu=cu).items():
        _close(r[name], want, TOL_GRAD, name)
    assert gdn.gdn_get_last_device_error() == 0


@pytest.mark.parametrize("B,T,H,Hk,d,W,S,ends", [
    (1, 1200, 4, 2, 64, 30, 3, list(range(0, 1200, 20)) + [1200]),                                   # a block for both heads
    (1, 900, 6, 2, 64, 40, 5, [0, 300, 301, 420, 420, 500, 557, 600, 640, 700, 760, 800, 900]),      # of three, one and two
    (3, 900, 5, 1, 128, 100, 3, None),                                                               # of five, four pieces
    (2, 1300, 8, 1, 64, 1300, 0, None),
], ids=str)
def test_gradients_of_shared_heads(B, T, H, Hk, d, W, S, ends):
    """A key head's query heads in one block and spread over several, evenly or
    not, with and without first tokens."""
    rng = np.random.default_rng(B + T + H)
    a = {n: _round(rng.standard_normal((B, T, h, d)), BF) for n, h in (("q", H), ("k", Hk), ("v", Hk), ("g", H))}
    t = {n: _dev(x, BF) for n, x in a.items()}
    kw = dict(window=W, sinks=S, cu_seqlens=_ints(ends))
    out, lse = attention.window_attention_fwd(t["q"], t["k"], t["v"], save_for_backward=True, **kw)
    r = attention.window_attention_bwd(t["q"], t["k"], t["v"], out, lse, t["g"], **kw)
    for n, want in A.window_bwd(a["q"], a["k"], a["v"], a["g"], W, S, cu=ends).items():
        _close(r[n], want, TOL_GRAD, n)
    again = attention.window_attention_bwd(t["q"], t["k"], t["v"], out, lse, t["g"], **kw)
    assert all(torch.equal(r[n], again[n]) for n in r)
    assert gdn.gdn_get_last_device_error() == 0


def test_malformed_offsets_are_recorded():
    """Out of order, beyond the row, not from zero: an error, and nothing outside the tensors is touched."""
    T = 300
    x = torch.randn(1, T, 64, device="cuda")
    q = torch.randn(1, T, 2, 64, device="cuda").to(BF)
    for cu in ([0, 200, 100, T], [0, 10, T + 50], [5, 100, T], [0, 100, 200], [0, -7, T], [0, 2 ** 31 - 1, T]):
        off = _ints(cu)
        calls = [lambda: mixer.gated_scan_fwd(x, x, x, x[0, 0], cu_seqlens=off),
                 lambda: attention.qk_norm_rope_fwd(q, q, inv_freq=torch.ones(32, device="cuda"), cu_seqlens=off),
                 lambda: attention.window_attention_fwd(q, q, q, 7, 1, cu_seqlens=off)]
        for call in calls:
            call()
            assert gdn.gdn_get_last_device_error() == 4, cu
        saved = mixer.gated_scan_fwd(x, x, x, x[0, 0], save_for_backward=True)[2]
        mixer.gated_scan_bwd(x, x, x, x[0, 0], x, saved, cu_seqlens=off)
        assert gdn.gdn_get_last_device_error() == 4, cu
        out, lse = attention.window_attention_fwd(q, q, q, 7, 1, save_for_backward=True)
        attention.window_attention_bwd(q, q, q, out, lse, q, 7, 1, cu_seqlens=off)
        assert gdn.gdn_get_last_device_error() == 4, cu
        cache = torch.zeros(len(cu), 8, 2, 64, device="cuda", dtype=BF)
        attention.window_cache_fill(q, q, cache, cache.clone(), sinks=1, cu_seqlens=off)
        assert gdn.gdn_get_last_device_error() == 4, cu


def test_rows_beyond_32_bits():
    """Rows 2^28 elements apart: the last ones start beyond 2^32."""
    T, step = 19, 1 << 28
    wide = torch.empty(T * step, dtype=BF, device="cuda").view(1, T, step)
    rng = np.random.default_rng(0)
    a = {k: _round(rng.standard_normal((1, T, 64)), BF) for k in "xri"}
    t = {}
    for n, k in enumerate("xri"):
        t[k] = wide[..., 64 * n:64 * n + 64]
        t[k].copy_(_dev(a[k], BF))
    lam = _round(rng.uniform(-5, -2, 64), F32)
    y, _, saved = mixer.gated_scan_fwd(t["x"], t["r"], t["i"], _dev(lam), save_for_backward=True)
    _close(y, M.gated_fwd(a["x"], a["r"], a["i"], lam)[0], TOL_BF16, "recurrence")
    dy = _round(rng.standard_normal((1, T, 64)), BF)
    g = mixer.gated_scan_bwd(t["x"], t["r"], t["i"], _dev(lam), _dev(dy, BF), saved)
    _close(g["dx"], M.gated_bwd(a["x"], a["r"], a["i"], lam, dy)["dx"], TOL_BF16, "dx")
    q, k, v = (t[n].unflatten(-1, (1, 64)) for n in "xri")
    na = {n: a[m][:, :, None] for n, m in zip("qkv", "xri")}
    out, lse = attention.window_attention_fwd(q, k, v, 4, 1, save_for_backward=True)
    _close(out, A.window_fwd(na["q"], na["k"], na["v"], 4, 1)[0], TOL_BF16, "attention")
    r = attention.window_attention_bwd(q, k, v, out, lse, _dev(dy, BF).unflatten(-1, (1, 64)), 4, 1)
    for n, want in A.window_bwd(na["q"], na["k"], na["v"], dy[:, :, None], 4, 1).items():
        _close(r[n], want, TOL_GRAD, n)
    tq, tk = attention.qk_norm_rope_fwd(q, k)
    _close(tq, A.rope_fwd(na["q"], None, None, None), TOL_BF16, "norm")
    _close(tk, A.rope_fwd(na["k"], None, None, None), TOL_BF16, "norm")
    assert gdn.gdn_get_last_device_error() == 0


def test_caches_beyond_32_bits():
    """Slots whose rows lie beyond 2^32 elements of the caches."""
    S, R, Hk, d, sinks = 70, 65000, 8, 128, 3
    kc, vc = (torch.empty(S, R, Hk, d, dtype=BF, device="cuda") for _ in range(2))
    slots, lengths = [S - 1, 68, 0], [50, R + 17, 120]
    assert (S - 1) * R * Hk * d > 2 ** 32
    rng = np.random.default_rng(1)
    q, k, v = (_round(rng.standard_normal((3, h, d)), BF) for h in (8, Hk, Hk))
    gen = torch.Generator(device="cuda").manual_seed(0)
    for s in slots:
        for c in (kc, vc):
            c[s] = torch.randn(R, Hk, d, generator=gen, device="cuda").to(BF)
    want = []
    for b, (s, n) in enumerate(zip(slots, lengths)):
        kk, vv = kc[s].double(), vc[s].double()
        at = A.cache_row(n, R - sinks, sinks)
        kk[at], vv[at] = torch.from_numpy(k[b]).cuda(), torch.from_numpy(v[b]).cuda()
        m = min(n + 1, R)
        w = torch.softmax(torch.einsum("hd,jhd->hj", torch.from_numpy(q[b]).cuda(), kk[:m]) / d ** 0.5, -1)
        want.append(_np(torch.einsum("hj,jhd->hd", w, vv[:m])))
    out = attention.window_attention_step(_dev(q, BF), _dev(k, BF), _dev(v, BF), kc, vc, _ints(lengths), sinks=sinks, slots=_ints(slots))
    _close(out, np.stack(want), TOL_BF16, "out")
    for b, (s, n) in enumerate(zip(slots, lengths)):
        at = A.cache_row(n, R - sinks, sinks)
        assert torch.equal(kc[s, at], _dev(k[b], BF)) and torch.equal(vc[s, at], _dev(v[b], BF))
    more = torch.randn(1, 40, Hk, d, generator=gen, device="cuda").to(BF)
    attention.window_cache_fill(more, more, kc, vc, sinks=sinks, slots=_ints([S - 1]))
    assert torch.equal(kc[S - 1, :40], more[0]) and torch.equal(vc[S - 1, :40], more[0])
    assert gdn.gdn_get_last_device_error() == 0


def test_calls_side_by_side_repeat_bit_for_bit():
    """Two streams at once, ten times: the results of one call alone."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF)  # noqa: E731
    x, r, i, dy, lam = n(1, 3000, 512), n(1, 3000, 512), n(1, 3000, 512), n(1, 3000, 512), -torch.rand(512, device="cuda") * 3 - 2
    q, k, v, g = n(2, 700, 4, 64), n(2, 700, 2, 64), n(2, 700, 2, 64), n(2, 700, 4, 64)

    def both():
        y, fs, saved = mixer.gated_scan_fwd(x, r, i, lam, save_for_backward=True)
        a = mixer.gated_scan_bwd(x, r, i, lam, dy, saved)
        out, lse = attention.window_attention_fwd(q, k, v, 200, 4, save_for_backward=True)
        b = attention.window_attention_bwd(q, k, v, out, lse, g, 200, 4)
        return [y, fs, *a.values(), out, lse, *b.values()]

    want = both()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        made = []
        for s in streams:
            with torch.cuda.stream(s):
                made.append(both())
        torch.cuda.synchronize()
        for got in made:
            assert all(torch.equal(x1, x2) for x1, x2 in zip(got, want))


def test_sequences_do_not_touch_each_other():
    """A neighbour's values, however large, change no bit of a packed sequence:
    of its outputs, its states or its gradients."""
    cu, T = [0, 100, 250, 411], 411
    gen = torch.Generator(device="cuda").manual_seed(8)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(BF)  # noqa: E731
    ins = [n(1, T, 4, 64), n(1, T, 2, 64), n(1, T, 2, 64), n(1, T, 4, 64)]
    seq = [n(1, T, 66) for _ in range(4)]
    lam, f = -torch.rand(66, device="cuda") * 3 - 2, 10000.0 ** (-torch.arange(32, device="cuda") / 32)

    def everything(q, k, v, g, x, r, i, dy):
        q, k = attention.qk_norm_rope_fwd(q, k, inv_freq=f, cu_seqlens=_ints(cu))
        q, k = q * big, k * big
        out, lse = attention.window_attention_fwd(q, k, v, 70, 3, cu_seqlens=_ints(cu), save_for_backward=True)
        b = attention.window_attention_bwd(q, k, v, out, lse, g, 70, 3, cu_seqlens=_ints(cu))
        y, fs, saved = mixer.gated_scan_fwd(x, r, i, lam, cu_seqlens=_ints(cu), save_for_backward=True)
        c = mixer.gated_scan_bwd(x, r, i, lam, dy, saved, cu_seqlens=_ints(cu))
        return [out, lse.transpose(1, 2), *b.values(), y, c["dx"], c["dr"], c["di"]], fs

    big = torch.ones(1, T, 1, 1, device="cuda", dtype=BF)
    want, states = everything(*ins, *seq)
    big[0, 100:250] = 64
    other = [t.clone() for t in (*ins, *seq)]
    for t in other:
        t[0, 100:250] *= 100
    got, new = everything(*other)
    for a, b in zip(got, want):
        assert torch.equal(a[0, :100], b[0, :100]) and torch.equal(a[0, 250:], b[0, 250:])
    assert torch.equal(new[0], states[0]) and torch.equal(new[2], states[2])


def test_queries_that_are_not_finite():
    """Their own outputs are NaN, and nobody else's."""
    q, k, v = (torch.randn(1, 4096, h, 64, device="cuda").to(BF) for h in (2, 2, 2))
    good = attention.window_attention_fwd(q, k, v, 4096)
    q[0, 1000:3000] = float("nan")
    out = attention.window_attention_fwd(q, k, v, 4096)
    assert torch.isnan(out[0, 1000:3000]).all()
    assert torch.equal(out[0, :1000], good[0, :1000]) and torch.equal(out[0, 3000:], good[0, 3000:])


def test_many_sequences_in_a_long_pack():
    """4096 sequences in 2^17 tokens: every operator that packs them, and of its
    results the sequences at the ends and some in between."""
    n, T, D = 4096, 1 << 17, 2048
    rng = np.random.default_rng(9)
    cu = np.concatenate([[0], np.sort(rng.choice(np.arange(1, T), n - 1, replace=False)), [T]])
    some = [0, 1, 1000, 2047, 3500, 4094, 4095]
    rows = np.concatenate([np.arange(cu[s], cu[s + 1]) for s in some])
    few = np.concatenate([[0], np.cumsum([cu[s + 1] - cu[s] for s in some])]).tolist()
    pick = lambda t: _np(t[:, torch.from_numpy(rows).cuda()])  # noqa: E731
    tc = _ints(cu)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r, i = (torch.randn(1, T, D, device="cuda", generator=gen).to(BF) for _ in range(3))
    lam = _round(rng.uniform(-4, -1, D), F32)
    h0, w = torch.randn(n, D, device="cuda", generator=gen), torch.randn(D, 4, device="cuda", generator=gen)
    y, fs = mixer.gated_scan_fwd(x, r, i, _dev(lam), initial_state=h0, cu_seqlens=tc)
    want, end = M.gated_fwd(pick(x), pick(r), pick(i), lam, h0=_np(h0[some]), cu=few)
    _close(torch.from_numpy(pick(y)), want, TOL_BF16, "recurrence")
    _close(fs[some], end, TOL_F32, "state")
    y, _ = mixer.short_conv_fwd(x, w, cu_seqlens=tc)
    alone, _ = mixer.short_conv_fwd(x[:, torch.from_numpy(rows).cuda()].contiguous(), w, cu_seqlens=_ints(few))
    assert np.array_equal(pick(y), _np(alone))
    q = x.view(1, T, 16, 128)
    k, v = (t.view(1, T, 16, 128)[:, :, :4].contiguous() for t in (r, i))
    out, lse = attention.window_attention_fwd(q, k, v, 20, 2, cu_seqlens=tc, save_for_backward=True)
    g = attention.window_attention_bwd(q, k, v, out, lse, q, 20, 2, cu_seqlens=tc)
    a = [pick(t) for t in (q, k, v)]
    _close(torch.from_numpy(pick(out)), A.window_fwd(*a, 20, 2, cu=few)[0], TOL_BF16, "attention")
    for name, want in A.window_bwd(*a, a[0], 20, 2, cu=few).items():
        _close(torch.from_numpy(pick(g[name])), want, TOL_GRAD, name)
    f = np.float32(10000.0) ** (-np.arange(64, dtype=np.float32) / 64)
    tq, _ = attention.qk_norm_rope_fwd(q, k, inv_freq=_dev(f), cu_seqlens=tc)
    _close(torch.from_numpy(pick(tq)), A.rope_fwd(a[0], None, f, A.positions_of(a[0], few)), TOL_BF16, "rotation")
    assert gdn.gdn_get_last_device_error() == 0


@pytest.mark.parametrize("B,T,H,Hk,d,W,S,cu", [
    (1, 700, 4, 2, 128, 200, 5, None),
    (2, 520, 3, 1, 64, 129, 33, None),   # two tiles of a head
    (1, 900, 2, 1, 64, 900, 0, None),    # the window is everything
    (1, 640, 2, 2, 128, 1, 3, None),     # itself and the first tokens
    (1, 800, 5, 1, 128, 70, 128, [0, 3, 300, 300, 431, 800]),
], ids=str)
def test_what_is_not_finite_reaches_its_readers_alone(B, T, H, Hk, d, W, S, cu):
    """Value by value: NaN and infinities of either sign at random places, each in a
    channel of its own or shared, and in whole rows.  An output is NaN, an infinity or
    its definition's number by what its token sees of that channel."""
    rng = np.random.default_rng(T + W)
    q, k, v = (_round(rng.standard_normal((B, T, h, d)), BF) for h in (H, Hk, Hk))
    bad = v.copy()
    for x in (np.nan, np.inf, -np.inf):
        for c in (0, 7, d - 1, *rng.integers(0, d, 3)):
            for n in range(3):
                bad[rng.integers(B), rng.integers(T), rng.integers(Hk), c] = x
    bad[0, -40] = np.nan
    bad[B - 1, T - 60, 0] = np.inf
    out, lse = attention.window_attention_fwd(_dev(q, BF), _dev(k, BF), _dev(bad, BF), W, S, cu_seqlens=_ints(cu), save_for_backward=True)
    want, want_lse = A.window_fwd(q, k, v, W, S, cu=cu)
    got, kind = _np(out), np.zeros(want.shape, int)  # 1: inf, 2: -inf, 3: both or a NaN
    for b, t0, t1 in A.rows_of(q, cu):
        i, j = np.arange(t1 - t0)[:, None], np.arange(t1 - t0)[None]
        see = ((j <= i) & ((i - j < W) | (j < S))).astype(float)
        for h in range(H):
            x = bad[b, t0:t1, h // (H // Hk)]
            nan, up, down = (see @ f.astype(float) > 0 for f in (np.isnan(x), x == np.inf, x == -np.inf))
            kind[b, t0:t1, h] = np.where(nan | (up & down), 3, np.where(up, 1, np.where(down, 2, 0)))
    assert np.array_equal(np.isnan(got), kind == 3) and np.array_equal(got == np.inf, kind == 1) and np.array_equal(got == -np.inf, kind == 2)
    assert (kind == 0).mean() > 0.2 and all((kind == x).any() for x in (1, 2, 3))
    fine = kind == 0
    _close(np.where(fine, got, 0), np.where(fine, want, 0), TOL_BF16, "the finite ones")
    _close(lse, want_lse, TOL_PAR, "lse")
    assert gdn.gdn_get_last_device_error() == 0


@pytest.mark.parametrize("W,S,places", [(4096, 0, [0]), (4096, 0, [5, 2000]), (512, 4, [5]), (4096, 0, slice(None)), (4096, 0, slice(0, None, 300))],
                         ids=str)
def test_a_nan_does_not_slow_its_readers(W, S, places):
    """Outputs are formed again where a value that is not seen spoils them, not where
    one that is seen does: well below ten times the time of finite values, where
    walking over every reader's keys took a thousand times it."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(1, 8192, h, 128, device="cuda", generator=gen).to(BF) for h in (16, 4, 4))
    bad = v.clone()
    bad[0, places, :, 3] = float("nan")

    def ms(x):
        best = float("inf")
        for _ in range(3):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            attention.window_attention_fwd(q, k, x, W, S)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    assert ms(bad) < 10 * ms(v)


def test_a_nan_behind_the_first_tokens_stays_near():
    """The block of first tokens is as wide as a multiple of 32: what else lies in it
    has no part in the gradients of queries that are far away, nor in their outputs."""
    rng = np.random.default_rng(5)
    W, S, T = 100, 4, 900
    a = {n: _round(rng.standard_normal((1, T, h, 64)), BF) for n, h in (("q", 4), ("k", 2), ("v", 2), ("g", 4))}
    t = {n: _dev(x, BF) for n, x in a.items()}
    for n in "kv":
        t[n][0, S:32] = float("nan")
    out, lse = attention.window_attention_fwd(t["q"], t["k"], t["v"], W, S, save_for_backward=True)
    r = attention.window_attention_bwd(t["q"], t["k"], t["v"], out, lse, t["g"], W, S)
    far = slice(31 + W + 254, None)
    _close(out[:, far], A.window_fwd(a["q"], a["k"], a["v"], W, S)[0][:, far], TOL_BF16, "out")
    _close(r["dq"][:, far], A.window_bwd(a["q"], a["k"], a["v"], a["g"], W, S)["dq"][:, far], TOL_GRAD, "dq")
    assert gdn.gdn_get_last_device_error() == 0
