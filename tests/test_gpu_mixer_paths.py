"""Paths of the mixer operators beyond the sizes of test_gpu_mixer.py, whose
inputs, comparisons and tolerances these tests use."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import gdn, mixer  # noqa: E402
from oracle import mixer as M  # noqa: E402
from tests import test_gpu_mixer as G  # noqa: E402

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def test_an_input_dropped_during_a_call_on_another_stream():
    """Its memory is not given out again while that stream still has to read it."""
    s = torch.cuda.Stream()
    want = mixer.group_norm_fwd(torch.ones(1237, 2048, device="cuda"), activation="none")
    x = torch.ones(1237, 2048, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
    at = x.data_ptr()
    y = mixer.group_norm_fwd(x, activation="none", stream=s)
    del x
    new = torch.empty(1237, 2048, device="cuda")
    assert not s.query() and new.data_ptr() != at
    s.synchronize()
    assert torch.equal(y, want)


def test_every_call_refuses_another_device(monkeypatch):
    """With device 1 said to be current, nothing on device 0 is launched."""
    x, w, h = torch.ones(2, 8, 16, device="cuda"), torch.ones(16, 4, device="cuda"), torch.ones(2, 3, 16, device="cuda")
    A, B = -torch.ones(16, 8, device="cuda"), torch.ones(2, 8, 1, 8, device="cuda")
    state = torch.ones(2, 16, 8, device="cuda")
    _, _, saved = mixer.ssm_scan_fwd(x, x, A, B, B, save_for_backward=True)
    monkeypatch.setattr(mixer, "_device", lambda: 1)
    for call in (lambda: mixer.short_conv_fwd(x, w), lambda: mixer.short_conv_bwd(x, w, x),
                 lambda: mixer.short_conv_step(x[:, 0], h, w),
                 lambda: mixer.ssm_scan_fwd(x, x, A, B, B), lambda: mixer.ssm_scan_bwd(x, x, A, B, B, x, saved),
                 lambda: mixer.ssm_scan_step(x[:, 0], x[:, 0], A, B[:, 0], B[:, 0], state),
                 lambda: mixer.group_norm_fwd(x), lambda: mixer.group_norm_bwd(x, x)):
        with pytest.raises(ValueError, match="current device is cuda:1"):
            call()


def test_second_derivatives_are_refused():
    x = torch.randn(2, 8, 16, device="cuda", requires_grad=True)
    w, A = torch.randn(16, 4, device="cuda"), -torch.ones(16, 8, device="cuda")
    B = torch.randn(2, 8, 1, 8, device="cuda")
    for f in (lambda: mixer.short_conv(x, w)[0], lambda: mixer.ssm_scan(x, x, A, B, B)[0], lambda: mixer.group_norm(x)):
        g, = torch.autograd.grad(f().sum(), x, create_graph=True)
        plain, = torch.autograd.grad(f().sum(), x)
        assert torch.equal(g, plain)
        with pytest.raises(RuntimeError, match="cannot be differentiated again"):
            (g.sum() + (x ** 3).sum()).backward()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_gradients_and_states_at_any_address(dtype):
    """Joined outputs hand slices of one gradient back, and a state may be a row
    of a cache: with odd widths neither starts at a 16-byte boundary."""
    D, N = 1003, 8
    xs = [torch.randn(1, 5, D, device="cuda").to(dtype).requires_grad_() for _ in range(2)]
    w = torch.randn(D, 4, device="cuda")
    A = -torch.rand(D, N, device="cuda")
    B = torch.randn(1, 5, 1, N, device="cuda").to(dtype)
    tail = torch.randn(3, 3, D, device="cuda").to(dtype)
    joined = torch.randn(D + 1, device="cuda")
    assert tail[1:2].data_ptr() % 16 and joined[1:].data_ptr() % 16
    for f in (lambda x: mixer.short_conv(x, w, joined[1:], initial_state=tail[1:2])[0],
              lambda x: mixer.ssm_scan(x, x, A, B, B, D=joined[1:])[0],
              lambda x: mixer.group_norm(x, joined[1:])):
        d = torch.randn(1, 10, D, device="cuda").to(dtype)
        assert d[:, 5:].data_ptr() % 16
        got = torch.autograd.grad(torch.cat([f(x) for x in xs], 1), xs, d)
        want = [torch.autograd.grad(f(x), x, d[:, 5 * i:5 * i + 5].clone())[0] for i, x in enumerate(xs)]
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    y, _ = mixer.short_conv_fwd(xs[0], w, initial_state=tail[1:2])
    y1, _ = mixer.short_conv_fwd(xs[0], w, initial_state=tail[1:2].clone())
    assert torch.equal(y, y1)


def test_a_scan_without_gradients_takes_no_memory_for_them():
    u = torch.randn(1, 256, 64, device="cuda", requires_grad=True)
    A, B = -torch.rand(64, 128, device="cuda"), torch.randn(1, 256, 1, 128, device="cuda")
    kept, _ = mixer.ssm_scan(u, u, A, B, B)
    grown = []
    for call in (lambda: mixer.ssm_scan_fwd(u, u, A, B, B), lambda: mixer.ssm_scan(u, u, A, B, B)):
        with torch.no_grad():
            torch.cuda.reset_peak_memory_stats()
            before = torch.cuda.memory_allocated()
            out, _ = call()
            grown.append(torch.cuda.max_memory_allocated() - before)
        assert torch.equal(out, kept) and not out.requires_grad
        del out
    assert grown[0] == grown[1]


# Sizes at which the kernels' loops turn more than once.  The tolerances of
# test_gpu_mixer.py hold: sums over n rows go through partial sums of at most 128
# tokens or a few rows per thread, whose roundings add up to about sqrt(n) 2^-24
# of the terms, as large a part of a sum that cancels down to sqrt(n) of them:
# 2^-24 x 30 for a thousand rows per partial sum, below the bounds for parameters.

NORM_ROWS = [  # rows, C, groups, strided: gradients of teams that take two to five rows
    (700, 2048, 16, False),  # a half warp per group (bf16), a warp (fp32)
    (500, 4096, 8, False),   # a warp with two vectors, 128 lanes
    (700, 2048, 2, False),   # 128 lanes with one vector
    (331, 4096, 1, False),   # a block per group
    (700, 2048, 1, True),    # 128 lanes; rows that no wide access fits
    (650, 2000, 8, False),   # groups of 250: two channels at a time in bf16
    (650, 1998, 6, True),    # groups of 333, one at a time
    (160, 8192, 1, False),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", NORM_ROWS, ids=str)
def test_norm_gradients_over_rows(case, dtype):
    rows, C, groups, _ = case
    teams = gdn.load().gdn_norm_bwd_workspace_size(10 ** 6, C, groups, int(dtype == F32)) // (8 * C)
    assert teams < rows / 1.05, "some team takes a second row"
    G.test_norm(case, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", [(1219, 2048, 16, False), (2433, 2048, 16, False), (1219, 2048, 8, False),
                                  (2437, 1024, 1, False), (2437, 512, 1, False)], ids=str)
def test_norm_of_several_rows_per_team(case, dtype):
    """Forwards of more teams than the GPU holds at a time: four rows each, the
    last ones fewer."""
    G.test_norm(case, dtype)


CONV_LONG = [  # B, T, D, W, cu, initial state, strided: blocks of 16 to 128 tokens
    (1, 12813, 1024, 4, None, True, False),
    (1, 3307, 1001, 4, None, True, False),
    (1, 6611, 1002, 3, None, False, False),
    (1, 3307, 1004, 2, [0, 1000, 1003, 1003, 3300, 3307], True, True),
    (2, 8203, 2048, 4, None, False, False),
    (1, 12813, 1024, 4, [0, 5, 6001, 6001, 12813], True, False),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CONV_LONG, ids=str)
def test_long_conv(case, dtype):
    G.test_conv(case, dtype)


SCAN_WIDE = [  # several blocks of 32 channels per group, the last one partly filled
    (2, 40, 70, 1, 16, None, True, False, True, True),
    (1, 50, 132, 2, 16, None, True, True, True, True),
    (1, 45, 100, 1, 8, None, False, False, False, True),
    (1, 64, 300, 3, 8, [0, 20, 20, 64], True, False, True, False),
    (1, 130, 262, 1, 16, [0, 1, 100, 130], True, False, True, True),
]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", SCAN_WIDE, ids=str)
def test_scan_of_several_channel_blocks(case, dtype):
    G._scan_check(case, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,D,G_,N,strided", [(77, 2048, 1, 16, False), (77, 2047, 1, 16, True), (39, 500, 2, 128, False)])
@pytest.mark.parametrize("with_slots", [False, True])
def test_scan_step_of_two_rows_per_thread(dtype, B, D, G_, N, strided, with_slots):
    """An odd number of rows, the last one alone; idle rows beside busy ones."""
    assert B * D * (N // 4) >= 152 * 2048 * 2 and B % 2
    a, t = G._scan_inputs((1, B, D, G_, N, None, False, strided, True, True), dtype)
    x = {k: t[k][0] for k in ("u", "dt", "z", "B", "C")}
    rng = np.random.default_rng(B)
    S = B + 3
    cache = G._round(rng.standard_normal((S, D, N)), F32)
    slots = rng.permutation(S)[:B]
    slots[[1, 4, B - 2]] = -1
    if not with_slots:
        slots = np.arange(B)
    state = G._dev(cache)
    sl = torch.tensor(slots, dtype=torch.int32, device="cuda") if with_slots else None
    y = mixer.ssm_scan_step(x["u"], x["dt"], t["A"], x["B"], x["C"], state, t["D"], x["z"], t["bias"], slots=sl)
    busy = np.flatnonzero(slots >= 0)
    rows = lambda k: np.moveaxis(a[k], 0, 1)[busy]  # one token of each row  # noqa: E731
    o, f = M.scan_fwd(rows("u"), rows("dt"), a["A"], rows("B"), rows("C"), a["D"], rows("z"), a["bias"], True,
                      cache[slots[busy]])
    want, new = np.zeros((B, D)), cache.copy()
    want[busy], new[slots[busy]] = o[:, 0], f
    G._close(y, want, G._io_tol(dtype, G.TOL_SCAN), "out")
    G._close(state, new, G.TOL_SCAN, "cache")
    G._no_device_error()


# Infinities beside the rows: slices of wider tensors whose other columns are
# infinite, at the addresses and strides of every copy width.

def _beside_infinity(a, dtype, left, right):
    flat = a.reshape(a.shape[0], a.shape[1], -1)
    wide = np.full(flat.shape[:-1] + (left + flat.shape[-1] + right,), np.inf, np.float32)
    wide[..., left:left + flat.shape[-1]] = flat
    t = G._dev(wide, dtype)[..., left:left + flat.shape[-1]]
    return t if a.ndim == 3 else t.unflatten(-1, a.shape[-2:])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("D", [40, 38, 37])
@pytest.mark.parametrize("left,right", [(8, 8), (2, 2), (3, 2)])  # 16-byte, 4-byte (bf16) and single elements
def test_infinities_beside_the_rows(dtype, D, left, right):
    right += -D % 8  # strides that the widest copies take where the left edge does
    case = (1, 100, D, 1, 16, [0, 40, 41, 100], True, False, True, True)
    a, t = G._scan_inputs(case, dtype)
    x = {k: _beside_infinity(a[k], dtype, left, right) for k in ("u", "dt", "z", "B", "C")}
    kw = dict(D=t["D"], z=x["z"], dt_bias=t["bias"], initial_state=t["h"], cu_seqlens=t["cu"])
    ref = (a["D"], a["z"], a["bias"], True, a["h"], case[5])
    args = (x["u"], x["dt"], t["A"], x["B"], x["C"])
    out, fs, saved = mixer.ssm_scan_fwd(*args, save_for_backward=True, **kw)
    o_ref, fs_ref = M.scan_fwd(a["u"], a["dt"], a["A"], a["B"], a["C"], *ref)
    tol = G._io_tol(dtype, G.TOL_SCAN)
    G._close(out, o_ref, tol, "out")
    G._close(fs, fs_ref, G.TOL_SCAN, "final_state")
    r = mixer.ssm_scan_bwd(*args, t["dout"], saved, **kw)
    want = M.scan_bwd(a["u"], a["dt"], a["A"], a["B"], a["C"], a["dout"], *ref)
    for k, v in r.items():
        G._close(v, want[k], G.TOL_SCAN_PAR if k in ("dA", "dD", "ddt_bias") else
                 G.TOL_SCAN if k == "d_initial_state" else tol, k)
    one = {k: v[0, 40:44] for k, v in x.items()}  # four rows of one token
    y = mixer.ssm_scan_step(one["u"], one["dt"], t["A"], one["B"], one["C"], torch.zeros(4, D, 16, device="cuda"),
                            t["D"], one["z"], t["bias"])
    rows = lambda k: np.moveaxis(a[k], 0, 1)[40:44]  # noqa: E731
    G._close(y, M.scan_fwd(rows("u"), rows("dt"), a["A"], rows("B"), rows("C"), a["D"], rows("z"), a["bias"])[0][:, 0],
             tol, "step")
    w = G._round(np.random.default_rng(D).uniform(-0.6, 0.6, (D, 4)), F32)
    tol = G._io_tol(dtype, G.TOL_F32)
    y, _ = mixer.short_conv_fwd(x["u"], G._dev(w), cu_seqlens=t["cu"])
    G._close(y, M.conv_fwd(a["u"], w, cu=case[5])[0], tol, "y")
    r = mixer.short_conv_bwd(x["u"], G._dev(w), t["dout"], cu_seqlens=t["cu"])
    want = M.conv_bwd(a["u"], w, a["dout"], cu=case[5])
    G._close(r["dx"], want["dx"], tol, "dx")
    G._close(r["dweight"], want["dweight"], G.TOL_PAR, "dweight")
    y = mixer.short_conv_step(one["u"], torch.zeros(4, 3, D, dtype=dtype, device="cuda"), G._dev(w))
    G._close(y, M.conv_fwd(rows("u"), w)[0][:, 0], tol, "step")
    n = mixer.group_norm_fwd(x["u"], gate=x["z"])
    G._close(n[0], M.norm_fwd(a["u"][0], gate=a["z"][0]), tol, "norm")
    r = mixer.group_norm_bwd(x["u"], t["dout"], gate=x["z"])
    want = M.norm_bwd(a["u"][0], a["dout"][0], gate=a["z"][0])
    for k, v in r.items():
        G._close(v[0], want[k], tol, k)
    G._no_device_error()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_stays_in_its_sequence_of_a_segmented_scan(value):
    """One input of the middle sequence, forward and back, where sequences run
    over several segments and start inside them."""
    cu = [0, 411, 700, 1100]
    case = (1, 1100, 24, 1, 16, cu, True, False, True, True)
    whole = 4 * (1100 * 2 * 16 + 3 * 24 * 18) + 512  # the reverse mode's partial sums without segments
    assert gdn.load().gdn_ssm_fwd_workspace_size(3, 1100, 24, 1, 16, 1) > 6 * 4 * 24 * 16
    assert gdn.load().gdn_ssm_bwd_workspace_size(3, 1100, 24, 1, 16, 1) > whole + 6 * 4 * 24 * 16
    a, t = G._scan_inputs(case, F32)
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["bias"], initial_state=t["h"], cu_seqlens=t["cu"])
    args = (t["dt"], t["A"], t["B"], t["C"])
    u = t["u"].clone()
    u[0, 500] = value
    (out, fs, saved), (out2, fs2, saved2) = (mixer.ssm_scan_fwd(x, *args, save_for_backward=True, **kw) for x in (t["u"], u))
    g, g2 = (mixer.ssm_scan_bwd(x, *args, t["dout"], s, d_final_state=t["dfs"], **kw) for x, s in ((t["u"], saved), (u, saved2)))
    assert torch.isnan(out2[0, 500]).all() if value != value else not torch.isfinite(out2[0, 500]).all()
    for rows in (slice(0, 411), slice(700, 1100)):
        for p, q in ((out, out2),) + tuple((g[k], g2[k]) for k in ("du", "ddt", "dz", "dB", "dC")):
            assert torch.equal(p[0, rows], q[0, rows])
    for n in (0, 2):
        assert torch.equal(fs[n], fs2[n]) and torch.equal(g["d_initial_state"][n], g2["d_initial_state"][n])
    assert torch.equal(out[0, 411:500], out2[0, 411:500])
    G._no_device_error()
