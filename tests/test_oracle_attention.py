"""The fp64 definitions of the gated recurrence and the attention operators
against closed forms, one another and central differences."""

import numpy as np
import pytest

from oracle import attention as A
from oracle import mixer as M

EPS = 1e-5  # central differences in fp64: error about EPS^2 + 1e-16 / EPS = 1e-10


def _check_gradient(f, args, grads, seed=0):
    rng = np.random.default_rng(seed)
    for name, a in args.items():
        d = rng.standard_normal(a.shape)
        ends = [f(**{**args, name: a + s * EPS * d}) for s in (1, -1)]
        want, got = (ends[0] - ends[1]) / (2 * EPS), float((grads[name] * d).sum())
        assert abs(got - want) <= 1e-7 * max(1.0, abs(want)), (name, got, want)


@pytest.mark.parametrize("cu", [None, [0, 0, 1, 4, 6]])
def test_gated_gradients(cu):
    rng = np.random.default_rng(1)
    B, T, D = (1 if cu else 2), 6, 3
    N = len(cu) - 1 if cu else B
    a = dict(x=rng.standard_normal((B, T, D)), r=rng.standard_normal((B, T, D)), i=rng.standard_normal((B, T, D)),
             lam=rng.uniform(-3, 1, D), h0=rng.standard_normal((N, D)))
    cy, cs = rng.standard_normal((B, T, D)), rng.standard_normal((N, D))

    def f(x, r, i, lam, h0):
        y, fs = M.gated_fwd(x, r, i, lam, 4.0, h0, cu)
        return float((y * cy).sum() + (fs * cs).sum())

    g = M.gated_bwd(a["x"], a["r"], a["i"], a["lam"], cy, 4.0, a["h0"], cu, cs)
    _check_gradient(f, a, {k: g["d_initial_state" if k == "h0" else "d" + k] for k in a})


def test_gated_closed_forms():
    """Open gates and a constant decay: a geometric sum; a closed decay gate: the state stays."""
    T, D = 7, 2
    lam, x = np.array([-1.0, 0.5]), np.ones((1, T, D))
    a = np.exp(-8.0 * np.logaddexp(0, lam) / 2)  # sigmoid(0) = 1/2
    y, fs = M.gated_fwd(x, np.zeros_like(x), np.full_like(x, 800.0), lam)
    for t in range(T):
        np.testing.assert_allclose(y[0, t], np.sqrt(1 - a * a) * (1 - a ** (t + 1)) / (1 - a), rtol=1e-12)
    y, fs = M.gated_fwd(x, np.full_like(x, -800.0), x, lam, h0=np.array([[3.0, -2.0]]))
    np.testing.assert_array_equal(fs, [[3.0, -2.0]])


@pytest.mark.parametrize("nxt", [False, True])
def test_rotation_gradients(nxt):
    rng = np.random.default_rng(2)
    x, w, g = rng.standard_normal((2, 3, 2, 32)), rng.uniform(0.5, 1.5, 32), rng.standard_normal((2, 3, 2, 32))
    f, pos = np.float32([1.0, 0.1, 0.01, 0.001]), rng.integers(0, 1000, (2, 3))
    dx, dw = A.rope_bwd(x, w, f, pos, g, interleaved=nxt)
    _check_gradient(lambda x, w: float((A.rope_fwd(x, w, f, pos, interleaved=nxt) * g).sum()), dict(x=x, w=w), dict(x=dx, w=dw))


def test_rotation_is_a_rotation():
    """Norms stay, scores depend on the distance alone, and angles of far positions are those of the exact product."""
    rng = np.random.default_rng(3)
    x, y = rng.standard_normal((1, 1, 1, 32)), rng.standard_normal((1, 1, 1, 32))
    f = np.float32(10000.0) ** (-np.arange(16, dtype=np.float32) / 16)
    at = lambda v, p: A.rope_fwd(v, None, f, np.array([[p]]), 0.0)[0, 0, 0]  # noqa: E731
    np.testing.assert_allclose(np.square(at(x, 977)).mean(), 1.0, rtol=1e-12)
    np.testing.assert_allclose(at(x, 1005) @ at(y, 1000), at(x, 5) @ at(y, 0), rtol=1e-10)
    angle = A._angles(np.array([[2 ** 30]]), np.float32([1.0]))[0, 0, 0, 0]
    exact = (2 ** 30 * 10 ** 30) % (2 * 3141592653589793238462643383279) / 10 ** 30  # pi to 31 digits
    assert abs(angle - exact) <= 1e-9


@pytest.mark.parametrize("cu", [None, [0, 0, 1, 5, 9]])
@pytest.mark.parametrize("W,S", [(1, 0), (3, 0), (3, 2), (50, 1)])
def test_window_gradients(cu, W, S):
    rng = np.random.default_rng(W + S)
    B, T = (1, 9) if cu else (2, 7)
    a = dict(q=rng.standard_normal((B, T, 4, 3)), k=rng.standard_normal((B, T, 2, 3)), v=rng.standard_normal((B, T, 2, 3)))
    g = rng.standard_normal((B, T, 4, 3))
    r = A.window_bwd(a["q"], a["k"], a["v"], g, W, S, cu=cu)
    _check_gradient(lambda q, k, v: float((A.window_fwd(q, k, v, W, S, cu=cu)[0] * g).sum()), a, {n: r["d" + n] for n in a})


def test_window_sees_what_it_says():
    """Each token's output as a sum over an explicit list of keys; the log-sum-exp; the step on a cache."""
    rng = np.random.default_rng(5)
    T, W, S = 23, 5, 3
    q, k, v = (rng.standard_normal((1, T, h, 4)) for h in (2, 1, 1))
    out, lse = A.window_fwd(q, k, v, W, S)
    kc, vc = (np.full((1, S + W, 1, 4), np.nan) for _ in range(2))
    for t in range(T):
        keys = sorted({j for j in range(t + 1) if j < S or t - j < W})
        assert len(keys) == min(t + 1, S + min(W, max(t + 1 - S, 0)))
        for h in range(2):
            s = k[0, keys, 0] @ q[0, t, h] / 2
            np.testing.assert_allclose(lse[0, h, t], np.log(np.exp(s).sum()), rtol=1e-12)
            np.testing.assert_allclose(out[0, t, h], np.exp(s) @ v[0, keys, 0] / np.exp(s).sum(), rtol=1e-12)
        o, kc, vc = A.window_step(q[:, t], k[:, t], v[:, t], kc, vc, [t], S)
        np.testing.assert_allclose(o[0], out[0, t], rtol=1e-12)


def test_broken_definitions_fail():
    """A window one too wide, a first token too few, a cache row taken modulo the wrong number."""
    rng = np.random.default_rng(6)
    q, k, v = (rng.standard_normal((1, 20, 2, 4)) for _ in range(3))
    good = A.window_fwd(q, k, v, 5, 2)[0]
    for W, S in ((6, 2), (4, 2), (5, 1), (5, 3)):
        assert np.abs(A.window_fwd(q, k, v, W, S)[0] - good).max() > 1e-2
    rows = [A.cache_row(p, 5, 2) for p in range(30)]
    assert all(sorted(rows[p - 4:p + 1]) == [2, 3, 4, 5, 6] for p in range(6, 30))  # the last five tokens, each in its row
    assert any(sorted(p % 7 for p in range(t - 4, t + 1)) != [2, 3, 4, 5, 6] for t in range(6, 30))
