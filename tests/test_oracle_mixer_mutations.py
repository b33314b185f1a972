"""The closed forms and differences that pin the fp64 mixer definitions fail
when a definition is broken (the mistake is planted in the oracle)."""

import numpy as np
import pytest

from oracle import mixer as M
from tests import test_oracle_mixer as P

conv_fwd, scan_fwd, scan_bwd, norm_fwd, norm_bwd = M.conv_fwd, M.scan_fwd, M.scan_bwd, M.norm_fwd, M.norm_bwd


def _backwards(x, w, *a, **k):
    return conv_fwd(x, w[:, ::-1], *a, **k)


def _no_state(x, w, bias=None, kind="silu", state=None, cu=None):
    return conv_fwd(x, w, bias, kind, None, cu)


def _growing(u, dt, A, *a, **k):
    return scan_fwd(u, dt, -A, *a, **k)


def _decay_after_write(u, dt, A, B, C, D=None, z=None, dt_bias=None, soft=True, state=None, cu=None, keep=None):
    """h <- a (h + x B)."""
    _, step = M._step(dt, dt_bias, soft)
    nb, T, d = u.shape
    y, fs = np.zeros_like(u), []
    for n, (b, t0, t1) in enumerate(M.bounds(nb, T, cu)):
        h = np.zeros(A.shape) if state is None else state[n]
        for t in range(t0, t1):
            if keep is not None:
                keep[(n, t)] = h
            Bt, Ct = (np.repeat(v[b, t], d // v.shape[2], axis=0) for v in (B, C))
            h = np.exp(step[b, t][:, None] * A) * (h + (step[b, t] * u[b, t])[:, None] * Bt)
            y[b, t] = (h * Ct).sum(1)
        fs.append(h)
    y = y if D is None else y + D * u
    return (y if z is None else y * M.act(z, "silu")), np.stack(fs)


def _no_skip_gradient(*a, **k):
    r = scan_bwd(*a, **k)
    return dict(r, dD=0 * r["dD"])


def _never_centered(*a, center=False, **k):
    return norm_fwd(*a, center=False, **k)


def _slightly_off(x, dy, w=None, *a, **k):
    r = norm_bwd(x, dy, w, *a, **k)
    return dict(r, dx=r["dx"] + 1e-3 * x)


@pytest.mark.parametrize("name,broken,pin", [
    ("conv_fwd", _backwards, lambda: P.test_conv_is_numpy_convolution()),
    ("conv_fwd", _backwards, lambda: P.test_conv_gradients(None, 4, "silu")),
    ("conv_fwd", _no_state, lambda: P.test_conv_gradients([0, 0, 1, 4, 6], 4, "silu")),
    ("scan_fwd", _growing, lambda: P.test_scan_closed_forms()),
    ("scan_fwd", _decay_after_write, lambda: P.test_scan_gradients(None, True, True)),
    ("scan_fwd", _decay_after_write, lambda: P.test_scan_gradients([0, 0, 1, 5], False, False)),
    ("scan_bwd", _no_skip_gradient, lambda: P.test_scan_gradients(None, True, True)),
    ("norm_fwd", _never_centered, lambda: P.test_norm_gradients("silu", True, False, True)),
    ("norm_bwd", _slightly_off, lambda: P.test_norm_gradients("none", False, False, False)),
])
def test_a_broken_definition_fails_its_pins(monkeypatch, name, broken, pin):
    pin()
    monkeypatch.setattr(M, name, broken)
    with pytest.raises(AssertionError):
        pin()
