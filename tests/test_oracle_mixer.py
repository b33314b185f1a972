"""The fp64 mixer definitions against closed forms and central differences."""

import numpy as np
import pytest

from oracle import mixer as M

EPS = 1e-5  # central differences in fp64: error about EPS^2 + 1e-16 / EPS = 1e-10


def _check_gradient(f, args, grads, seed=0):
    """Directional derivatives of sum(f) along random directions."""
    rng = np.random.default_rng(seed)
    for name, a in args.items():
        d = rng.standard_normal(a.shape)
        up, down = dict(args), dict(args)
        up[name], down[name] = a + EPS * d, a - EPS * d
        want = (f(**up) - f(**down)) / (2 * EPS)
        got = float((grads[name] * d).sum())
        assert abs(got - want) <= 1e-7 * max(1.0, abs(want)), (name, got, want)


@pytest.mark.parametrize("cu", [None, [0, 0, 1, 4, 6]])
@pytest.mark.parametrize("W,kind", [(2, "none"), (3, "silu"), (4, "silu")])
def test_conv_gradients(cu, W, kind):
    rng = np.random.default_rng(W)
    B, T, D = (1 if cu else 2), 6, 3
    N = len(cu) - 1 if cu else B
    a = dict(x=rng.standard_normal((B, T, D)), w=rng.standard_normal((D, W)), bias=rng.standard_normal(D),
             state=rng.standard_normal((N, W - 1, D)))
    cy, cs = rng.standard_normal((B, T, D)), rng.standard_normal((N, W - 1, D))

    def f(x, w, bias, state):
        y, fs = M.conv_fwd(x, w, bias, kind, state, cu)
        return float((y * cy).sum() + (fs * cs).sum())

    r = M.conv_bwd(a["x"], a["w"], cy, a["bias"], kind, a["state"], cu, cs)
    _check_gradient(f, a, dict(x=r["dx"], w=r["dweight"], bias=r["dbias"], state=r["d_initial_state"]))


def test_conv_is_numpy_convolution():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((1, 9, 2)), rng.standard_normal((2, 4))
    y, fs = M.conv_fwd(x, w, None, "none")
    for d in range(2):
        np.testing.assert_allclose(y[0, :, d], np.convolve(x[0, :, d], w[d, ::-1])[:9], atol=1e-14)
    np.testing.assert_array_equal(fs[0], x[0, -3:])


@pytest.mark.parametrize("cu", [None, [0, 0, 1, 5]])
@pytest.mark.parametrize("gated,soft", [(True, True), (False, False)])
def test_scan_gradients(cu, gated, soft):
    rng = np.random.default_rng(3)
    B, T, D, G, N = (1 if cu else 2), 5, 4, 2, 3
    nseq = len(cu) - 1 if cu else B
    a = dict(u=rng.standard_normal((B, T, D)), dt=rng.uniform(0.1, 1, (B, T, D)), A=-rng.uniform(0.2, 2, (D, N)),
             Bm=rng.standard_normal((B, T, G, N)), Cm=rng.standard_normal((B, T, G, N)), D=rng.standard_normal(D),
             dt_bias=rng.uniform(0, 0.5, D), state=rng.standard_normal((nseq, D, N)))
    if gated:
        a["z"] = rng.standard_normal((B, T, D))
    cy, cs = rng.standard_normal((B, T, D)), rng.standard_normal((nseq, D, N))

    def f(u, dt, A, Bm, Cm, D, dt_bias, state, z=None):
        y, fs = M.scan_fwd(u, dt, A, Bm, Cm, D, z, dt_bias, soft, state, cu)
        return float((y * cy).sum() + (fs * cs).sum())

    r = M.scan_bwd(a["u"], a["dt"], a["A"], a["Bm"], a["Cm"], cy, a["D"], a.get("z"), a["dt_bias"], soft, a["state"],
                   cu, cs)
    g = dict(u=r["du"], dt=r["ddt"], A=r["dA"], Bm=r["dB"], Cm=r["dC"], D=r["dD"], dt_bias=r["ddt_bias"],
             state=r["d_initial_state"], z=r["dz"])
    _check_gradient(f, a, g)


def test_scan_closed_forms():
    """B = 0 is pure decay; A = 0 with unit inputs is a running sum."""
    rng = np.random.default_rng(4)
    T, D, N = 6, 2, 3
    dt, A, h0 = rng.uniform(0.1, 1, (1, T, D)), -rng.uniform(0.2, 2, (D, N)), rng.standard_normal((1, D, N))
    zero, one = np.zeros((1, T, 1, N)), np.ones((1, T, 1, N))
    _, fs = M.scan_fwd(np.ones((1, T, D)), dt, A, zero, one, soft=False, state=h0)
    np.testing.assert_allclose(fs[0], np.exp(dt[0].sum(0)[:, None] * A) * h0[0], rtol=1e-13)
    u = rng.standard_normal((1, T, D))
    y, _ = M.scan_fwd(u, np.ones((1, T, D)), 0 * A, one, one, soft=False)
    np.testing.assert_allclose(y, N * np.cumsum(u, 1), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("kind", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate,first", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("center", [False, True])
def test_norm_gradients(kind, gate, first, center):
    rng = np.random.default_rng(5)
    a = dict(x=rng.standard_normal((3, 8)), w=rng.standard_normal(8), b=rng.standard_normal(8))
    if gate:
        a["gate"] = rng.standard_normal((3, 8))
    cy = rng.standard_normal((3, 8))
    kw = dict(groups=2, kind=kind, center=center, gate_first=first)

    def f(x, w, b, gate=None):
        return float((M.norm_fwd(x, w, b, gate, **kw) * cy).sum())

    r = M.norm_bwd(a["x"], cy, a["w"], a["b"], a.get("gate"), **kw)
    _check_gradient(f, a, dict(x=r["dx"], w=r["dweight"], b=r["dbias"], gate=r.get("dgate")))


def test_a_planted_mistake_breaks_the_pins():
    """The decay applied after the write, and a window read backwards, are seen."""
    rng = np.random.default_rng(6)
    u, dt, A = rng.standard_normal((1, 4, 2)), rng.uniform(0.1, 1, (1, 4, 2)), -rng.uniform(0.5, 2, (2, 3))
    Bm, Cm = rng.standard_normal((1, 4, 1, 3)), rng.standard_normal((1, 4, 1, 3))
    y, _ = M.scan_fwd(u, dt, A, Bm, Cm, soft=False)
    h = np.zeros((2, 3))
    bad = np.zeros_like(u)
    for t in range(4):
        h = np.exp(dt[0, t][:, None] * A) * (h + (dt[0, t] * u[0, t])[:, None] * Bm[0, t])
        bad[0, t] = (h * Cm[0, t]).sum(1)
    assert np.abs(y - bad).max() > 1e-2
    w = rng.standard_normal((2, 4))
    assert np.abs(M.conv_fwd(u, w)[0] - M.conv_fwd(u, w[:, ::-1])[0]).max() > 1e-2
