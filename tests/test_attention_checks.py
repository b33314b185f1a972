"""Refusals of the gated recurrence and the attention operators: the wrappers'
checks (CPU tensors), the C ABI's host validation (addresses that are never
dereferenced), and what the wrappers do around a call."""

import ctypes
import math
import sys

import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import attention, build, gdn, mixer  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def _z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def _gated(**over):
    return {**dict(x=_z(2, 8, 12), r=_z(2, 8, 12), i=_z(2, 8, 12), lam=torch.zeros(12)), **over}


@pytest.mark.parametrize("over,msg", [
    (dict(x=_z(2, 8, 12, dtype=torch.float16)), "x must be"), (dict(x=_z(8, 12)), "x must be"),
    (dict(r=_z(2, 8, 12, dtype=F32)), "r must be"), (dict(i=_z(2, 8, 11)), "i must have shape"),
    (dict(lam=torch.zeros(11)), "lam must have shape"), (dict(lam=_z(12)), "lam must be"), (dict(rate=0.0), "rate"),
    (dict(rate=float("nan")), "rate"), (dict(rate=float("inf")), "rate"), (dict(initial_state=torch.zeros(2, 11)), "initial_state"),
    (dict(initial_state=_z(2, 12)), "initial_state"), (dict(cu_seqlens=torch.tensor([0, 8], dtype=torch.int32)), "batch extent 1"),
    ({}, "CUDA"),
])
def test_gated_refusals(over, msg):
    with pytest.raises(ValueError, match=msg):
        mixer.gated_scan_fwd(**_gated(**over))


def test_gated_step_refusals():
    row, lam = [_z(4, 12)] * 3, torch.zeros(12)
    for state, msg in ((torch.zeros(3, 12), "a row for each"), (torch.zeros(4, 11), "state must be"), (_z(4, 12), "state must be")):
        with pytest.raises(ValueError, match=msg):
            mixer.gated_scan_step(*row, lam, state)
    with pytest.raises(ValueError, match="slots must be"):
        mixer.gated_scan_step(*row, lam, torch.zeros(3, 12), slots=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="out_state must have shape"):
        mixer.gated_scan_step(*row, lam, torch.zeros(4, 12), out_state=torch.zeros(5, 12))


def _rope(**over):
    return {**dict(q=_z(2, 8, 4, 64), k=_z(2, 8, 2, 64), q_weight=torch.zeros(64), k_weight=torch.zeros(64),
                   inv_freq=torch.zeros(32)), **over}


@pytest.mark.parametrize("over,msg", [
    (dict(q=_z(2, 8, 256)), "q and k must be"), (dict(q=_z(2, 8, 4, 64, dtype=torch.float16)), "q must be"),
    (dict(k=_z(2, 8, 2, 32)), "k must have shape"), (dict(k=_z(2, 7, 2, 64)), "k must have shape"),
    (dict(k=_z(2, 8, 2, 64, dtype=F32)), "k must be"), (dict(q=_z(2, 8, 4, 96), k=_z(2, 8, 2, 96)), "head size"),
    (dict(q_weight=torch.zeros(32)), "q_weight"), (dict(k_weight=_z(64)), "k_weight"),
    (dict(inv_freq=torch.zeros(36)), "inv_freq"), (dict(inv_freq=torch.zeros(6)), "inv_freq"),
    (dict(inv_freq=torch.zeros(32, dtype=torch.float64)), "inv_freq must be"),
    (dict(positions=torch.zeros(2, 8, dtype=torch.int64)), "positions must be"),
    (dict(positions=torch.zeros(8, dtype=torch.int32)), "positions must have shape"),
    (dict(cu_seqlens=torch.tensor([0, 8], dtype=torch.int32)), "batch extent 1"),
    (dict(q=_z(2, 4, 8, 64).transpose(1, 2)), "dense rows"), ({}, "CUDA"),
])
def test_rotation_refusals(over, msg):
    with pytest.raises(ValueError, match=msg):
        attention.qk_norm_rope_fwd(**_rope(**over))


def test_frequencies_have_no_gradient():
    with pytest.raises(ValueError, match="inv_freq has no gradient"):
        attention.qk_norm_rope(**_rope(inv_freq=torch.zeros(32, requires_grad=True)))


def _window(**over):
    return {**dict(q=_z(2, 8, 4, 64), k=_z(2, 8, 2, 64), v=_z(2, 8, 2, 64), window=4), **over}


@pytest.mark.parametrize("over,msg", [
    (dict(q=_z(8, 4, 64)), "q and k must be"), (dict(q=_z(2, 8, 4, 64, dtype=F32)), "q must be"),
    (dict(k=_z(2, 8, 2, 128)), "k must have shape"), (dict(k=_z(2, 9, 2, 64)), "k must have shape"),
    (dict(v=_z(2, 8, 1, 64)), "v must have shape"), (dict(v=_z(2, 8, 2, 64, dtype=F32)), "v must be"),
    (dict(q=_z(2, 8, 4, 96), k=_z(2, 8, 2, 96), v=_z(2, 8, 2, 96)), "head size"),
    (dict(k=_z(2, 8, 3, 64), v=_z(2, 8, 3, 64)), "divide into"), (dict(window=0), "window"), (dict(window=-1), "window"),
    (dict(sinks=-1), "sinks"), (dict(sinks=129), "sinks"), (dict(scale=0.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    ({}, "CUDA"),
])
def test_window_refusals(over, msg):
    with pytest.raises(ValueError, match=msg):
        attention.window_attention_fwd(**_window(**over))


class Library:
    """Notes what a call hands to the library."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 256

        def call(*args):
            held = [v for v in sys._getframe(1).f_locals.values() if isinstance(v, torch.Tensor)]
            held += [t for v in sys._getframe(1).f_locals.values() if isinstance(v, list) for t in v if isinstance(t, torch.Tensor)]
            self.calls.append((name, args, held))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    made = Library()
    for m in (mixer, attention):
        monkeypatch.setattr(m, "load", lambda: made)
        monkeypatch.setattr(m, "_on_gpu", lambda dev, x: None)
        monkeypatch.setattr(m, "_current", lambda dev: 0)
    return made


def test_step_refusals(fake):
    q, k, caches, lengths = _z(3, 4, 64), _z(3, 2, 64), (_z(3, 9, 2, 64), _z(3, 9, 2, 64)), torch.zeros(3, dtype=torch.int32)
    step = attention.window_attention_step
    step(q, k, k, *caches, lengths, sinks=2)
    (name, args, _), = fake.calls
    assert name == "gdn_window_step" and args[11:18] == (3, 3, 4, 2, 64, 7, 2)
    for bad, msg in ((dict(sinks=9), "sinks . window"), (dict(k_cache=_z(3, 9, 2, 128)), "k_cache|alike"),
                     (dict(k_cache=_z(2, 9, 2, 64), v_cache=_z(2, 9, 2, 64)), "2 rows for a batch of 3"),
                     (dict(v_cache=_z(3, 8, 2, 64)), "alike"), (dict(lengths=lengths.long()), "lengths must be"),
                     (dict(lengths=lengths[:2]), "lengths must have shape"), (dict(slots=lengths[:2]), "slots must have shape"),
                     (dict(k_cache=_z(3, 2, 9, 64).transpose(1, 2)), "contiguous"), (dict(k_cache=_z(3, 9, 2, 64, dtype=F32)), "k_cache must be"),
                     (dict(k_cache=_off(3, 9, 2, 64)), "16-byte")):
        kw = {**dict(k_cache=caches[0], v_cache=caches[1], lengths=lengths, sinks=2), **bad}
        with pytest.raises(ValueError, match=msg):
            step(q, k, k, kw.pop("k_cache"), kw.pop("v_cache"), kw.pop("lengths"), **kw)
    fill = attention.window_cache_fill
    fill(_z(2, 30, 2, 64), _z(2, 30, 2, 64), *caches, sinks=2)
    assert fake.calls[-1][0] == "gdn_window_fill" and fake.calls[-1][1][8:15] == (2, 30, 3, 2, 64, 7, 2)
    with pytest.raises(ValueError, match="3 rows for 4 sequences"):
        fill(_z(4, 30, 2, 64), _z(4, 30, 2, 64), *caches, sinks=2)
    with pytest.raises(ValueError, match="slots must have shape"):
        fill(_z(4, 30, 2, 64), _z(4, 30, 2, 64), *caches, sinks=2, slots=lengths)
    assert len(fake.calls) == 2


def _off(*shape, dtype=BF):
    """A contiguous tensor that starts where no 16-byte access fits."""
    n = math.prod(shape)
    t = torch.randn(n + 64).to(dtype)[1:1 + n].view(shape)
    assert t.is_contiguous() and t.data_ptr() % 16
    return t


def _f32(*shape):
    return _off(*shape, dtype=F32)


CALLS = {
    "gated_fwd": (lambda **t: mixer.gated_scan_fwd(_z(2, 4, 5), _z(2, 4, 5), _z(2, 4, 5), **t),
                  dict(lam=_f32(5), initial_state=_f32(2, 5))),
    "gated_bwd": (lambda **t: mixer.gated_scan_bwd(_z(2, 4, 5), _z(2, 4, 5), _z(2, 4, 5), t.pop("lam"), t.pop("d_out"),
                                                   torch.zeros(256, dtype=torch.uint8), **t),
                  dict(lam=_f32(5), initial_state=_f32(2, 5), d_out=_off(2, 4, 5), d_final_state=_f32(2, 5))),
    "gated_step": (lambda **t: mixer.gated_scan_step(_z(2, 5), _z(2, 5), _z(2, 5), t["lam"], torch.zeros(2, 5)), dict(lam=_f32(5))),
    "rope_fwd": (lambda **t: attention.qk_norm_rope_fwd(_z(2, 3, 2, 32), _z(2, 3, 1, 32), **t),
                 dict(q_weight=_f32(32), k_weight=_f32(32), inv_freq=_f32(8))),
    "rope_bwd": (lambda **t: attention.qk_norm_rope_bwd(_z(2, 3, 2, 32), _z(2, 3, 1, 32), **t),
                 dict(dq_out=_off(2, 3, 2, 32), dk_out=_off(2, 3, 1, 32), q_weight=_f32(32), k_weight=_f32(32), inv_freq=_f32(8))),
    "window_fwd": (lambda **t: attention.window_attention_fwd(window=3, **t),
                   dict(q=_off(2, 3, 2, 64), k=_off(2, 3, 1, 64), v=_off(2, 3, 1, 64))),
    "window_bwd": (lambda **t: attention.window_attention_bwd(window=3, **t),
                   dict(q=_off(2, 3, 2, 64), k=_off(2, 3, 1, 64), v=_off(2, 3, 1, 64), out=_off(2, 3, 2, 64), lse=_f32(2, 2, 3),
                        d_out=_off(2, 3, 2, 64))),
    "window_step": (lambda **t: attention.window_attention_step(**t, k_cache=_z(2, 5, 1, 64), v_cache=_z(2, 5, 1, 64),
                                                                lengths=torch.zeros(2, dtype=torch.int32)),
                    dict(q=_off(2, 2, 64), k=_off(2, 1, 64), v=_off(2, 1, 64))),
    "window_fill": (lambda **t: attention.window_cache_fill(**t, k_cache=_z(2, 5, 1, 64), v_cache=_z(2, 5, 1, 64)),
                    dict(k=_off(2, 3, 1, 64), v=_off(2, 3, 1, 64))),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_inputs_at_any_address(fake, name):
    """What the library reads 16 bytes at a time it gets at a 16-byte boundary, as
    a copy that the caller holds; what is there already is handed on as it is."""
    call, inputs = CALLS[name]
    call(**inputs)
    _, args, held = fake.calls[-1]
    at = [a for a in args if isinstance(a, int) and a > 1 << 20]
    assert at and not [a for a in at if a % 16]
    for k, t in inputs.items():
        assert any(h.data_ptr() in at and h.shape == t.shape and torch.equal(h, t) for h in held), k
    there = {k: t.clone() for k, t in inputs.items()}
    call(**there)
    at = [a for a in fake.calls[-1][1] if isinstance(a, int) and a > 1 << 20]
    assert all(t.data_ptr() in at for t in there.values())


def test_slices_of_one_projection_are_read_where_they_are(fake):
    qkv = torch.randn(2, 7, (4 + 2 + 2) * 64).to(BF)
    q, k, v = (t.unflatten(-1, (-1, 64)) for t in qkv.split([256, 128, 128], -1))
    attention.window_attention_fwd(q, k, v, 3)
    args = fake.calls[-1][1]
    assert args[:6] == (q.data_ptr(), 512, k.data_ptr(), 512, v.data_ptr(), 512)
    attention.qk_norm_rope_fwd(q, k)
    assert fake.calls[-1][1][:4] == (q.data_ptr(), 512, k.data_ptr(), 512)
    odd = torch.randn(2, 7, 515).to(BF)[..., :512].split([256, 128, 128], -1)  # rows no 16-byte piece fits
    attention.window_attention_fwd(*(t.unflatten(-1, (-1, 64)) for t in odd), 3)
    args = fake.calls[-1][1]
    assert args[1::2][:3] == (256, 128, 128) and not [a for a in args[:6:2] if a % 16]


def test_a_window_beyond_the_row_is_the_row(fake):
    attention.window_attention_fwd(_z(1, 9, 2, 64), _z(1, 9, 2, 64), _z(1, 9, 2, 64), 1 << 40, 3)
    assert fake.calls[-1][1][14:16] == (9, 3)


OPERATORS = {
    "gated": (lambda x, w: mixer.gated_scan(x, x.detach(), x.detach(), w)[0], mixer, "gated_scan",
              lambda x, *a, **k: (x * x, x.sum(1), x.new_zeros(4)),
              lambda x, r, i, lam, d, *a, **k: dict(dx=2 * x * d, dr=0 * r, di=0 * i, dlam=0 * lam)),
    "rope": (lambda x, w: attention.qk_norm_rope(x, x.detach(), w)[0], attention, "qk_norm_rope",
             lambda q, k, *a, **kw: (q * q, k + 0),
             lambda q, k, d, dk, w, *a, **kw: dict(dq=2 * q * d, dk=0 * k, dq_weight=0 * w)),
    "window": (lambda x, w: attention.window_attention(x, x.detach(), x.detach() + 0 * w.sum(), 3), attention, "window_attention",
               lambda q, *a, save_for_backward=False, **kw: (q * q, q.sum(-1)) if save_for_backward else q * q,
               lambda q, k, v, o, s, d, *a, **kw: dict(dq=2 * q * d, dk=0 * k, dv=0 * v)),
}


@pytest.mark.parametrize("name", list(OPERATORS))
def test_first_derivatives_only(monkeypatch, name):
    f, module, prefix, fwd, bwd = OPERATORS[name]
    monkeypatch.setattr(module, prefix + "_fwd", fwd)
    monkeypatch.setattr(module, prefix + "_bwd", bwd)
    x, w = torch.randn(2, 5, 4, requires_grad=True), torch.randn(4, requires_grad=True)
    g, gw = torch.autograd.grad(f(x, w).sum(), (x, w), create_graph=True)
    assert torch.equal(g, 2 * x) and not gw.any()
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        (g.sum() + (x ** 3).sum()).backward()
    f(x, w).sum().backward()
    assert torch.equal(x.grad, 2 * x)


def test_nothing_is_kept_where_no_backward_can_follow(monkeypatch):
    saves = []

    def fwd(x, *a, save_for_backward=False, **kw):
        saves.append(save_for_backward)
        return (x + 0, None, x) if save_for_backward else (x + 0, None)

    monkeypatch.setattr(mixer, "gated_scan_fwd", fwd)
    monkeypatch.setattr(attention, "window_attention_fwd",
                        lambda q, *a, save_for_backward=False, **kw: (saves.append(save_for_backward), (q + 0, q) if save_for_backward else q + 0)[1])
    for f, names in ((lambda **t: mixer.gated_scan(**t)[0], ("x", "r", "i", "lam", "initial_state")),
                     (lambda **t: attention.window_attention(**t, window=2), ("q", "k", "v"))):
        a = {k: torch.zeros(2) for k in names}
        assert not f(**a).requires_grad and not saves[-1]
        for k in names:
            leaf = {**a, k: torch.zeros(2, requires_grad=True)}
            assert f(**leaf).requires_grad and saves[-1], k
            with torch.no_grad():
                assert not f(**leaf).requires_grad and not saves[-1], k


# ------------------------------------------------------------------- the C ABI

def test_gated_host_validation(lib):
    def call(x=FAKE, xs=64, r=FAKE, rs=64, i=FAKE, i_s=64, lam=FAKE, rate=8.0, h=None, cu=None, y=FAKE, fs=None, saved=None, n=0,
             B=1, T=20, D=64, dtype=0):
        return lib.gdn_gated_fwd(x, xs, r, rs, i, i_s, lam, rate, h, cu, y, fs, saved, n, B, T, D, dtype, None)
    assert call(B=0) == 1 and call(T=-1) == 1 and call(D=0) == 1 and call(dtype=2) == 1 and call(B=70000) == 2 and call(D=70000) == 2
    assert call(x=None) == 1 and call(r=None) == 1 and call(i=None) == 1 and call(lam=None) == 1 and call(y=None) == 1
    assert call(xs=63) == 1 and call(rs=63) == 1 and call(i_s=63) == 1 and call(rate=0.0) == 1 and call(rate=float("nan")) == 1 and call(rate=float("inf")) == 1
    assert call(x=FAKE + 1) == 3 and call(r=FAKE + 2, dtype=1) == 3 and call(lam=FAKE + 4) == 3 and call(y=FAKE + 2) == 3
    assert call(cu=FAKE + 2) == 3 and call(h=FAKE, fs=FAKE) == 1 and call(T=0) == 0
    need = lib.gdn_gated_saved_size(1, 20, 64, 0)
    assert need == 3 * 64 * 4 and lib.gdn_gated_saved_size(5, 20, 64, 1) == need and lib.gdn_gated_saved_size(0, 20, 64, 0) == 0
    assert call(saved=FAKE, n=need - 1) == 1 and call(saved=FAKE + 16, n=need) == 3
    wneed = lib.gdn_gated_bwd_workspace_size(1, 20, 64, 0)
    assert wneed > 0 and lib.gdn_gated_bwd_workspace_size(1, 20, 0, 0) == 0

    def bwd(saved=FAKE, n=need, ws=FAKE, wn=wneed, dx=FAKE, dlam=FAKE, d0=None, dfs=None, d_out=FAKE):
        return lib.gdn_gated_bwd(FAKE, 64, FAKE, 64, FAKE, 64, FAKE, 8.0, None, None, d_out, dfs, saved, n, dx, FAKE, FAKE, dlam, d0,
                                 1, 20, 64, 0, ws, wn, None)
    assert bwd(saved=None) == 1 and bwd(n=need - 1) == 1 and bwd(ws=None) == 1 and bwd(wn=wneed - 1) == 1 and bwd(ws=FAKE + 16) == 3
    assert bwd(dx=None) == 1 and bwd(dlam=None) == 1 and bwd(d_out=None) == 1 and bwd(dx=FAKE + 2) == 3 and bwd(d0=FAKE, dfs=FAKE) == 1

    def step(S=4, slots=None, state=FAKE, B=4):
        return lib.gdn_gated_step(FAKE, 64, FAKE, 64, FAKE, 64, FAKE, 8.0, state, FAKE, slots, FAKE, B, S, 64, 0, None)
    assert step(S=3) == 1 and step(S=0, slots=FAKE) == 1 and step(state=None) == 1 and step(slots=FAKE + 2) == 3


def test_rotation_host_validation(lib):
    def call(q=FAKE, qs=256, k=FAKE, ks=128, w=FAKE, f=FAKE, pos=None, cu=None, qo=FAKE, ko=FAKE, B=1, T=8, H=4, Hk=2, d=64, n=32, dtype=0):
        return lib.gdn_rope_fwd(q, qs, k, ks, w, w, f, pos, cu, qo, ko, B, T, H, Hk, d, n, 0, 1e-6, dtype, None)
    assert call(T=0) == 0  # nothing to do
    assert call(H=0) == 1 and call(Hk=0) == 1 and call(n=-4) == 1 and call(d=96) == 2 and call(n=6) == 2 and call(n=36) == 1
    assert call(H=1025, qs=1025 * 64) == 2 and call(B=0) == 1 and call(dtype=5) == 1 and call(B=40000, T=60000) == 2
    assert call(q=None) == 1 and call(k=None) == 1 and call(f=None) == 1 and call(qo=None) == 1 and call(ko=None) == 1
    assert call(qs=255) == 1 and call(ks=127) == 1 and call(q=FAKE + 1) == 3 and call(f=FAKE + 4) == 3 and call(qo=FAKE + 8) == 3
    assert call(pos=FAKE + 2) == 3 and call(cu=FAKE + 1) == 3
    need = lib.gdn_rope_bwd_workspace_size(1, 8, 4, 2, 64, 0)
    assert need > 0 and lib.gdn_rope_bwd_workspace_size(1, 8, 4, 2, 48, 0) == 0

    def bwd(w=FAKE, dw=FAKE, g=FAKE, dq=FAKE, ws=FAKE, n=need):
        return lib.gdn_rope_bwd(FAKE, 256, FAKE, 128, w, None, FAKE, None, None, g, FAKE, dq, FAKE, dw, None, 1, 8, 4, 2, 64, 32, 0,
                                1e-6, 0, ws, n, None)
    assert bwd(dw=None) == 1 and bwd(w=None) == 1 and bwd(g=None) == 1 and bwd(dq=None) == 1
    assert bwd(ws=None) == 1 and bwd(n=need - 1) == 1 and bwd(ws=FAKE + 64) == 3 and bwd(dq=FAKE + 2) == 3


def test_window_host_validation(lib):
    def call(q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, cu=None, out=FAKE, lse=None, B=1, T=8, H=4, Hk=2, d=64, W=4, S=0, scale=0.1):
        return lib.gdn_window_fwd(q, qs, k, ks, v, vs, cu, out, lse, B, T, H, Hk, d, W, S, scale, None)
    assert call(T=0) == 0  # nothing to do
    assert call(H=0) == 1 and call(Hk=3) == 1 and call(W=0) == 1 and call(S=-1) == 1 and call(scale=0.0) == 1 and call(scale=-1.0) == 1
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1 and call(d=96) == 2 and call(S=129) == 2
    assert call(H=2048, Hk=2) == 2 and call(B=70000) == 2 and call(B=60000, T=40000) == 2 and call(B=0) == 1 and call(T=-1) == 1
    assert call(q=None) == 1 and call(k=None) == 1 and call(v=None) == 1 and call(out=None) == 1
    assert call(qs=248) == 1 and call(ks=120) == 1 and call(vs=120) == 1 and call(qs=260) == 3 and call(vs=132) == 3
    assert call(q=FAKE + 8) == 3 and call(v=FAKE + 2) == 3 and call(out=FAKE + 8) == 3 and call(lse=FAKE + 4) == 3 and call(cu=FAKE + 2) == 3
    # delta alone where the window is everything, the first tokens' partial sums where it is not
    size = lib.gdn_window_bwd_workspace_size
    assert size(1, 1024, 4, 4, 64, 1024, 4, 0) == 4 * 4 * 1024 and size(1, 1024, 4, 4, 64, 100, 0, 0) == 4 * 4 * 1024
    assert size(1, 1024, 4, 4, 64, 128, 4, 0) == 4 * 4 * 1024 + 4 * 4 * 4 * 2 * 4 * 64  # stretches of two tiles: four
    # and those of a key head's two query heads, where they go to two blocks, but not where one is enough for the GPU
    heads = 4 * 2 * 1024 * 2 * 2 * 64
    assert size(1, 1024, 4, 2, 64, 1024, 4, 0) == 4 * 4 * 1024 + heads and size(1, 1024, 4, 2, 64, 100, 0, 0) == 4 * 4 * 1024 + heads
    assert size(1, 1024, 4, 2, 64, 128, 4, 0) == 4 * 4 * 1024 + 2 * 4 * 4 * 2 * 2 * 4 * 64 + heads
    assert size(8, 1024, 4, 2, 64, 100, 0, 0) == 8 * 4 * 4 * 1024
    assert size(1, 1000, 4, 3, 64, 100, 0, 0) == 0
    need = size(1, 8, 4, 2, 64, 4, 2, 0)

    def bwd(out=FAKE, lse=FAKE, g=FAKE, dq=FAKE, ws=FAKE, n=need):
        return lib.gdn_window_bwd(FAKE, 256, FAKE, 128, FAKE, 128, None, out, lse, g, dq, FAKE, FAKE, 1, 8, 4, 2, 64, 4, 2, 0.1, ws, n, None)
    assert bwd(out=None) == 1 and bwd(lse=None) == 1 and bwd(g=None) == 1 and bwd(dq=None) == 1 and bwd(dq=FAKE + 8) == 3
    assert bwd(ws=None) == 1 and bwd(n=need - 1) == 1 and bwd(ws=FAKE + 128) == 3

    def step(k=FAKE, kc=FAKE, ln=FAKE, slots=None, B=4, S=4, W=4, sinks=2, out=FAKE):
        return lib.gdn_window_step(FAKE, 256, k, 128, FAKE, 128, kc, FAKE, ln, slots, out, B, S, 4, 2, 64, W, sinks, 0.1, None)
    assert step(S=3) == 1 and step(S=0, slots=FAKE) == 1 and step(kc=None) == 1 and step(ln=None) == 1 and step(out=None) == 1
    assert step(W=0) == 1 and step(W=(1 << 30) + 1) == 2 and step(k=FAKE + 8) == 3 and step(kc=FAKE + 8) == 3 and step(ln=FAKE + 2) == 3
    assert step(slots=FAKE + 1) == 3

    def fill(k=FAKE, kc=FAKE, slots=None, B=2, S=2, T=9):
        return lib.gdn_window_fill(k, 128, FAKE, 128, None, slots, kc, FAKE, B, T, S, 2, 64, 4, 2, None)
    assert fill(T=0) == 0 and fill(S=1) == 1 and fill(kc=None) == 1 and fill(k=None) == 1 and fill(k=FAKE + 4) == 3 and fill(slots=FAKE + 2) == 3


def test_workspaces_of_long_rows(lib):
    """Sizes are counted in 64 bits."""
    assert lib.gdn_gated_saved_size(1, 1 << 28, 1024, 0) == (1 << 25) * 1024 * 4
    assert lib.gdn_window_bwd_workspace_size(1, 1 << 29, 16, 1, 64, 1 << 29, 0, 0) == 4 * 16 << 29
    assert ctypes.sizeof(ctypes.c_size_t) == 8


def test_packs_of_many_sequences(lib):
    """A packed call has N sequences in T tokens altogether: what limits a call is T,
    not N times T."""
    window, rope = lib.gdn_window_bwd_workspace_size, lib.gdn_rope_bwd_workspace_size
    for n, T in ((512, 1 << 20), (2048, 1 << 18), (4096, 1 << 17), (2048, 1 << 20), (65535, 1 << 20)):
        assert window(n, T, 16, 4, 128, 1024, 4, 1) > 0 and rope(n, T, 16, 4, 128, 1) > 0, (n, T)
        assert lib.gdn_gated_saved_size(n, T, 2048, 1) == T // 8 * 2048 * 4 and lib.gdn_gated_bwd_workspace_size(n, T, 2048, 1) > 0
        assert lib.gdn_conv_bwd_workspace_size(n, T, 2048, 4, 1) > 0 and lib.gdn_ssm_saved_size(n, T, 2048, 16, 1) > 0
        assert lib.gdn_ssm_bwd_workspace_size(n, T, 2048, 1, 16, 1) > 0
    # dense rows of as many tokens each are too many
    assert window(4096, 1 << 17, 16, 4, 128, 1024, 4, 0) == 0 and rope(2048, 1 << 20, 16, 4, 128, 0) == 0
    assert lib.gdn_gated_saved_size(4096, 1 << 17, 2048, 0) == 0 and lib.gdn_conv_bwd_workspace_size(4096, 1 << 17, 2048, 4, 0) == 0
    # and so is a pack that is too long by itself
    assert lib.gdn_gated_saved_size(1, 1 << 29, 65536, 1) == 0 and window(1, (1 << 30) + 1, 1, 1, 64, 9, 0, 1) == 0
    # the calls look at the same limit: a missing input is what they name
    N, T, cu = 4096, 1 << 17, FAKE
    assert lib.gdn_gated_fwd(None, 2048, FAKE, 2048, FAKE, 2048, FAKE, 8.0, None, cu, FAKE, None, None, 0, N, T, 2048, 0, None) == 1
    assert lib.gdn_rope_fwd(None, 2048, FAKE, 512, None, None, FAKE, None, cu, FAKE, FAKE, 2048, 1 << 20, 16, 4, 128, 64, 0, 1e-6, 0, None) == 1
    assert lib.gdn_window_fwd(None, 2048, FAKE, 512, FAKE, 512, cu, FAKE, None, N, T, 16, 4, 128, 1024, 4, 0.1, None) == 1
    assert lib.gdn_window_fill(None, 512, FAKE, 512, cu, None, FAKE, FAKE, N, T, N, 4, 128, 1024, 4, None) == 1
    assert lib.gdn_conv_fwd(FAKE, 2048, None, None, None, cu, FAKE, None, N, T, 2048, 4, 1, 0, None) == 1


FORWARD_MODE = {
    "gated": (lambda x, r, i, lam, h: mixer.gated_scan(x, r, i, lam, initial_state=h),
              dict(x=_z(2, 4, 8), r=_z(2, 4, 8), i=_z(2, 4, 8), lam=torch.zeros(8), h=torch.zeros(2, 8))),
    "ssm": (lambda u, dt, A, B, C, D, z, b, h: mixer.ssm_scan(u, dt, A, B, C, D, z, b, initial_state=h),
            dict(u=_z(2, 4, 8), dt=_z(2, 4, 8), A=torch.zeros(8, 8), B=_z(2, 4, 1, 8), C=_z(2, 4, 1, 8), D=torch.zeros(8), z=_z(2, 4, 8),
                 b=torch.zeros(8), h=torch.zeros(2, 8, 8))),
    "rope": (lambda q, k, w: attention.qk_norm_rope(q, k, w), dict(q=_z(2, 4, 2, 64), k=_z(2, 4, 1, 64), w=torch.zeros(64))),
    "window": (lambda q, k, v: attention.window_attention(q, k, v, 3), dict(q=_z(2, 4, 2, 64), k=_z(2, 4, 1, 64), v=_z(2, 4, 1, 64))),
}


@pytest.mark.parametrize("grad", [True, False], ids=["grad", "no_grad"])
@pytest.mark.parametrize("name", list(FORWARD_MODE))
def test_forward_mode_is_refused(fake, name, grad):
    """A dual tensor carries a derivative without requires_grad, under no_grad too: a
    result without a tangent would count as constant."""
    from torch.autograd import forward_ad
    f, inputs = FORWARD_MODE[name]
    with torch.set_grad_enabled(grad), forward_ad.dual_level():
        f(**inputs)  # (nothing asks for a derivative)
        for k, t in inputs.items():
            with pytest.raises(NotImplementedError, match="forward mode"):
                f(**{**inputs, k: forward_ad.make_dual(t, torch.ones_like(t))})
    f(**inputs)


def test_an_empty_batch_is_the_librarys_refusal(monkeypatch, lib):
    """Every form names the argument, none trips over the workspace that sizes like
    these do not have."""
    for m in (mixer, attention):
        monkeypatch.setattr(m, "_on_gpu", lambda dev, x: None)
        monkeypatch.setattr(m, "_current", lambda dev: 0)
    x, lam, byte = _z(0, 4, 8), torch.zeros(8), torch.zeros(0, dtype=torch.uint8)
    q, k, w = _z(0, 4, 2, 64), _z(0, 4, 1, 64), torch.zeros(64)
    lse = torch.zeros(0, 2, 4)
    for call in (lambda: mixer.gated_scan_fwd(x, x, x, lam), lambda: mixer.gated_scan_bwd(x, x, x, lam, x, byte),
                 lambda: mixer.gated_scan_step(x[:, 0], x[:, 0], x[:, 0], lam, torch.zeros(2, 8)),
                 lambda: mixer.short_conv_bwd(x, torch.zeros(8, 4), x),
                 lambda: mixer.ssm_scan_bwd(x, x, torch.zeros(8, 8), _z(0, 4, 1, 8), _z(0, 4, 1, 8), x, byte),
                 lambda: attention.qk_norm_rope_fwd(q, k, w), lambda: attention.qk_norm_rope_bwd(q, k, q, k, w),
                 lambda: attention.window_attention_fwd(q, k, k, 3), lambda: attention.window_attention_bwd(q, k, k, q, lse, q, 3),
                 lambda: attention.window_attention_step(q[:, 0], k[:, 0], k[:, 0], _z(2, 5, 1, 64), _z(2, 5, 1, 64), torch.zeros(0, dtype=torch.int32)),
                 lambda: attention.window_cache_fill(k, k, _z(2, 5, 1, 64), _z(2, 5, 1, 64))):
        with pytest.raises(gdn.GdnError, match="INVALID_ARG"):
            call()
