"""Refusals of the mixer operators: the wrappers' checks (CPU tensors) and the
C ABI's host validation (addresses that are never dereferenced)."""

import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import build, gdn, mixer  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gdn.load()


def _scan(**over):
    a = dict(u=torch.zeros(2, 8, 12, dtype=BF), dt=torch.zeros(2, 8, 12, dtype=BF), A=torch.zeros(12, 16),
             B=torch.zeros(2, 8, 2, 16, dtype=BF), C=torch.zeros(2, 8, 2, 16, dtype=BF), D=torch.zeros(12),
             z=torch.zeros(2, 8, 12, dtype=BF), dt_bias=torch.zeros(12))
    a.update(over)
    return a


@pytest.mark.parametrize("over,msg", [
    (dict(u=torch.zeros(2, 8, 12, dtype=torch.float16)), "u must be"),
    (dict(dt=torch.zeros(2, 8, 12)), "dt must be"),
    (dict(z=torch.zeros(2, 8, 11, dtype=BF)), "z must have shape"),
    (dict(A=torch.zeros(12, 24)), "state size"),
    (dict(A=torch.zeros(11, 16)), "A must be"),
    (dict(A=torch.zeros(12, 16, dtype=BF)), "A must be"),
    (dict(B=torch.zeros(2, 8, 16, dtype=BF)), "B must be"),
    (dict(B=torch.zeros(2, 8, 5, 16, dtype=BF)), "groups"),
    (dict(C=torch.zeros(2, 8, 1, 16, dtype=BF)), "C must have shape"),
    (dict(D=torch.zeros(13)), "D must have shape"),
    (dict(dt_bias=torch.zeros(12, dtype=BF)), "dt_bias must be"),
    (dict(u=torch.zeros(8, 12, dtype=BF)), "u must be"),
    (dict(initial_state=torch.zeros(2, 12, 16, dtype=BF)), "initial_state must be|CUDA"),
    (dict(cu_seqlens=torch.tensor([0, 8], dtype=torch.int32)), "batch extent 1"),
    (dict(cu_seqlens=torch.tensor([0, 8])), "int32"),
    ({}, "CUDA"),
])
def test_scan_refusals(over, msg):
    with pytest.raises(ValueError, match=msg):
        mixer.ssm_scan_fwd(**_scan(**over))


@pytest.mark.parametrize("x,w,kw,msg", [
    (torch.zeros(2, 8, 12, dtype=BF), torch.zeros(12, 5), {}, "taps"),
    (torch.zeros(2, 8, 12, dtype=BF), torch.zeros(11, 4), {}, "weight must be"),
    (torch.zeros(2, 8, 12, dtype=BF), torch.zeros(12, 4, dtype=BF), {}, "weight must be"),
    (torch.zeros(8, 12, dtype=BF), torch.zeros(12, 4), {}, "x must be"),
    (torch.zeros(2, 8, 12, dtype=BF), torch.zeros(12, 4), dict(activation="sigmoid"), "activation"),
    (torch.zeros(2, 8, 12, dtype=BF), torch.zeros(12, 4), dict(initial_state=torch.zeros(2, 3, 12)), "initial_state"),
    (torch.zeros(2, 8, 12, dtype=BF), torch.zeros(12, 4), dict(initial_state=torch.zeros(2, 4, 12, dtype=BF)),
     "initial_state"),
    (torch.zeros(2, 8, 12, dtype=BF), torch.zeros(12, 4), {}, "CUDA"),
])
def test_conv_refusals(x, w, kw, msg):
    with pytest.raises(ValueError, match=msg):
        mixer.short_conv_fwd(x, w, **kw)


@pytest.mark.parametrize("kw,msg", [
    (dict(groups=5), "groups"), (dict(weight=torch.zeros(8)), "weight"), (dict(gate=torch.zeros(4, 64)), "gate"),
    (dict(activation="gelu"), "activation"), ({}, "CUDA"),
])
def test_norm_refusals(kw, msg):
    with pytest.raises(ValueError, match=msg):
        mixer.group_norm_fwd(torch.zeros(4, 64, dtype=BF), **kw)


def test_step_refusals():
    x, w = torch.zeros(4, 12, dtype=BF), torch.zeros(12, 4)
    with pytest.raises(ValueError, match="a row for each"):
        mixer.short_conv_step(x, torch.zeros(3, 3, 12, dtype=BF), w)
    with pytest.raises(ValueError, match="state must be"):
        mixer.short_conv_step(x, torch.zeros(4, 2, 12, dtype=BF), w)
    with pytest.raises(ValueError, match="slots must be"):
        mixer.short_conv_step(x, torch.zeros(3, 3, 12, dtype=BF), w, slots=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="out_state must have shape"):
        mixer.short_conv_step(x, torch.zeros(4, 3, 12, dtype=BF), w, out_state=torch.zeros(5, 3, 12, dtype=BF))


def test_uneven_rows_are_refused():
    x = torch.zeros(4, 6, 16)
    rows = lambda t, inner=1: mixer._rows(t, t.shape[-1] * (t.shape[-2] if inner == 2 else 1), inner)[1]  # noqa: E731
    assert rows(x) == 16 and rows(x[..., 3:7]) == 16 and rows(x[:, :1]) == 96 and rows(x[:, :1, 2:9]) == 96
    assert rows(x[:1, ::2]) == 32 and rows(x[:, :, :8].unflatten(2, (2, 4)), 2) == 16
    for bad in (x[:, 1:], x.transpose(1, 2), x[..., ::2], x[:, :1].expand(4, 6, 16), x[:, ::2][:, :2]):
        with pytest.raises(ValueError):
            rows(bad)


def test_conv_host_validation(lib):
    def call(x=FAKE, stride=64, w=FAKE, y=FAKE, h=None, fs=None, cu=None, B=1, T=8, D=64, W=4, act=1, dtype=0):
        return lib.gdn_conv_fwd(x, stride, w, None, h, cu, y, fs, B, T, D, W, act, dtype, None)
    assert call(W=5) == 2 and call(W=1) == 2 and call(B=70000) == 2 and call(D=70000, stride=70000) == 2
    assert call(B=0) == 1 and call(T=-1) == 1 and call(D=0) == 1 and call(act=2) == 1 and call(dtype=2) == 1
    assert call(x=None) == 1 and call(w=None) == 1 and call(y=None) == 1 and call(stride=63) == 1
    assert call(x=FAKE + 1) == 3 and call(x=FAKE + 2, dtype=1) == 3 and call(y=FAKE + 2) == 3 and call(cu=FAKE + 2) == 3
    assert call(h=FAKE, fs=FAKE) == 1  # the final state over the initial one
    need = lib.gdn_conv_bwd_workspace_size(1, 8, 64, 4, 0)
    assert need > 0 and lib.gdn_conv_bwd_workspace_size(1, 8, 64, 7, 0) == 0

    def bwd(ws=FAKE, nbytes=need, dx=FAKE, dw=FAKE):
        return lib.gdn_conv_bwd(FAKE, 64, FAKE, None, None, None, FAKE, None, dx, dw, None, None, 1, 8, 64, 4, 1, 0,
                                ws, nbytes, None)
    assert bwd(ws=None) == 1 and bwd(nbytes=need - 1) == 1 and bwd(ws=FAKE + 16) == 3
    assert bwd(dx=None) == 1 and bwd(dw=None) == 1 and bwd(dx=FAKE + 2) == 3

    def step(S=4, slots=None, state=FAKE, B=4):
        return lib.gdn_conv_step(FAKE, 64, FAKE, None, state, FAKE, slots, FAKE, B, S, 64, 4, 1, 0, None)
    assert step(S=3) == 1 and step(S=0, slots=FAKE) == 1 and step(state=None) == 1 and step(slots=FAKE + 2) == 3


def test_scan_host_validation(lib):
    def call(u=FAKE, us=64, A=FAKE, b=FAKE, bs=32, z=FAKE, zs=64, out=FAKE, saved=None, sbytes=0, B=1, T=32, D=64, G=2,
             N=16, dtype=0):
        return lib.gdn_ssm_fwd(u, us, FAKE, 64, A, b, bs, FAKE, 32, None, z, zs, None, 1, None, None, out, None, saved,
                               sbytes, B, T, D, G, N, dtype, None, 0, None)
    assert call(N=24) == 2 and call(N=4) == 2 and call(G=3) == 1 and call(G=0) == 1 and call(T=-1) == 1
    assert call(u=None) == 1 and call(A=None) == 1 and call(b=None) == 1 and call(out=None) == 1
    assert call(us=63) == 1 and call(bs=31) == 1 and call(zs=10) == 1 and call(z=FAKE + 1) == 3
    assert call(A=FAKE + 4) == 3 and call(b=FAKE + 1) == 3 and call(dtype=7) == 1
    need = lib.gdn_ssm_saved_size(1, 32, 64, 16, 0)
    assert need == 4 * 64 * 16 * 4 and lib.gdn_ssm_saved_size(3, 32, 64, 16, 1) == (32 // 8 + 3) * 64 * 16 * 4
    assert lib.gdn_ssm_saved_size(1, 32, 64, 12, 0) == 0
    assert call(saved=FAKE, sbytes=need - 1) == 1 and call(saved=FAKE + 16, sbytes=need) == 3
    wneed = lib.gdn_ssm_bwd_workspace_size(1, 32, 64, 2, 16, 0)
    assert wneed > 0 and lib.gdn_ssm_bwd_workspace_size(1, 32, 64, 3, 16, 0) == 0

    def bwd(saved=FAKE, sbytes=need, z=None, dz=None, dA=FAKE, ws=FAKE, nbytes=wneed, du=FAKE):
        return lib.gdn_ssm_bwd(FAKE, 64, FAKE, 64, FAKE, FAKE, 32, FAKE, 32, None, z, 64, None, 1, None, FAKE, None,
                               saved, sbytes, du, FAKE, dz, FAKE, FAKE, dA, None, None, None, 1, 32, 64, 2, 16, 0, ws,
                               nbytes, None)
    assert bwd(saved=None) == 1 and bwd(sbytes=need - 1) == 1 and bwd(dA=None) == 1 and bwd(du=None) == 1
    assert bwd(z=FAKE) == 1 and bwd(dz=FAKE) == 1 and bwd(ws=None) == 1 and bwd(nbytes=wneed - 1) == 1
    assert bwd(ws=FAKE + 64) == 3 and bwd(du=FAKE + 8) == 3


def test_norm_host_validation(lib):
    def call(x=FAKE, xs=64, gate=None, gs=0, y=FAKE, rows=4, C=64, groups=2, act=1, dtype=0):
        return lib.gdn_norm_fwd(x, xs, gate, gs, None, None, y, rows, C, groups, 1e-6, act, 0, 0, dtype, None)
    assert call(rows=0) == 0  # nothing to do
    assert call(groups=3) == 1 and call(groups=0) == 1 and call(C=0) == 1 and call(rows=-1) == 1
    assert call(act=3) == 1 and call(dtype=2) == 1 and call(x=None) == 1 and call(y=None) == 1
    assert call(xs=32) == 1 and call(gate=FAKE, gs=63) == 1 and call(gate=FAKE + 1, gs=64) == 3 and call(y=FAKE + 8) == 3
    assert call(C=16386, xs=16386) == 2
    need = lib.gdn_norm_bwd_workspace_size(4, 64, 2, 0)
    assert need > 0

    def bwd(w=FAKE, dw=FAKE, gate=None, dgate=None, ws=FAKE, nbytes=need):
        return lib.gdn_norm_bwd(FAKE, 64, gate, 64, w, None, FAKE, FAKE, dgate, dw, None, 4, 64, 2, 1e-6, 1, 0, 0, 0,
                                ws, nbytes, None)
    assert bwd(dw=None) == 1 and bwd(w=None) == 1 and bwd(gate=FAKE) == 1 and bwd(dgate=FAKE) == 1
    assert bwd(ws=None) == 1 and bwd(nbytes=need - 1) == 1 and bwd(ws=FAKE + 32) == 3
