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
