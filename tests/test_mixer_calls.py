"""What the mixer wrappers do around a call, on the CPU: streams, devices,
gradients and addresses, with the kernels and the CUDA runtime replaced."""

import contextlib
import ctypes
import math
import sys
import types

import pytest

torch = pytest.importorskip("torch")

from torch.utils.checkpoint import checkpoint  # noqa: E402

from linear_attention_sequence_chunked_gb300 import build, gdn, mixer  # noqa: E402


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is a CUDA one and notes the streams that it is
    recorded on."""
    is_cuda = property(lambda self: True)

    def record_stream(self, stream):
        self.__dict__.setdefault("streams", []).append(stream)


def _on_gpu(*shape):
    return torch.zeros(*shape).as_subclass(OnGpu)


@pytest.mark.parametrize("kind", ["one", "pair", "dict"])
def test_tensors_of_a_call_on_another_stream_are_recorded(monkeypatch, kind):
    """Inputs, state caches among them, stay until the given stream is through
    with them, outputs until the caller's is."""
    stream = types.SimpleNamespace(device=torch.device("cuda", 0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("caller", device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    ins = dict(x=_on_gpu(2, 4), state=_on_gpu(2, 3), weight=_on_gpu(4), bias=None, eps=1e-6)
    outs = _on_gpu(2, 4), _on_gpu(2, 3)
    made = {"one": outs[0], "pair": (outs[0], None), "dict": dict(dx=outs[0], dweight=outs[1])}[kind]

    def call(**args):
        assert set(args) == set(ins)
        for k in ("x", "state", "weight"):  # whatever the call does, they are safe already
            assert args[k].streams == [stream], k
        return made

    assert mixer._on_stream(call, dict(ins, stream=stream)) is made
    assert outs[0].streams == [("caller", stream.device)]


def test_tensors_of_another_device_are_refused(monkeypatch):
    x = torch.zeros(2, 4)
    monkeypatch.setattr(mixer, "_device", lambda: 0, raising=False)
    mixer._on_gpu(0, x)
    with pytest.raises(ValueError, match="tensors are on cuda:1, the current device is cuda:0"):
        mixer._on_gpu(1, x)


def _square(x):
    """Its gradient 2 x d_out depends on x where d_out is a constant too."""
    return x * x


OPERATORS = {  # the operator as autograd sees it, and x^2 and 2 x d_out in its kernels' place
    "conv": (lambda x, w: mixer.short_conv(x, w)[0], "short_conv", lambda x, *a, **k: (_square(x), x[:, -3:].clone()),
             lambda x, w, d, *a, **k: dict(dx=2 * x * d, dweight=torch.zeros_like(w))),
    "scan": (lambda x, w: mixer.ssm_scan(x, x.detach(), w, x.detach(), x.detach())[0], "ssm_scan",
             lambda u, *a, **k: (_square(u), u.sum(1), u.new_zeros(4)),
             lambda u, dt, A, B, C, d, *a, **k: dict(du=2 * u * d, ddt=0 * u, dA=0 * A, dB=0 * B, dC=0 * C)),
    "norm": (lambda x, w: mixer.group_norm(x, w), "group_norm", lambda x, *a, **k: _square(x),
             lambda x, d, w, *a, **k: dict(dx=2 * x * d, dweight=torch.zeros_like(w))),
}


@pytest.mark.parametrize("name", list(OPERATORS))
def test_second_derivatives_are_refused(monkeypatch, name):
    """Where another path to the same input has a second derivative, only that
    one would come back."""
    f, prefix, fwd, bwd = OPERATORS[name]
    monkeypatch.setattr(mixer, prefix + "_fwd", fwd)
    monkeypatch.setattr(mixer, prefix + "_bwd", bwd)
    x, w = torch.randn(2, 5, 4, requires_grad=True), torch.randn(4, 4, requires_grad=True)
    g, gw = torch.autograd.grad(f(x, w).sum(), (x, w), create_graph=True)
    assert torch.equal(g, 2 * x) and not gw.any()
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        (g.sum() + (x ** 3).sum()).backward()
    f(x, w).sum().backward()  # the first derivative, as before
    assert torch.equal(x.grad, 2 * x)


def test_gradients_of_constants_can_be_used_in_a_graph(monkeypatch):
    """What does not reach the operator again is not refused."""
    f, prefix, fwd, bwd = OPERATORS["norm"]
    monkeypatch.setattr(mixer, prefix + "_fwd", fwd)
    monkeypatch.setattr(mixer, prefix + "_bwd", bwd)
    x, s = torch.randn(2, 5, 4, requires_grad=True), torch.tensor(3.0, requires_grad=True)
    g, = torch.autograd.grad(f(x, torch.ones(4)).sum(), x, create_graph=True)
    (s * g.detach()).sum().backward()
    assert torch.allclose(s.grad, (2 * x).sum())


class Library:
    """Notes the addresses that a call hands to the library, and the tensors
    that its caller holds meanwhile."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 256

        def call(*args):
            held = {k: v for k, v in sys._getframe(1).f_locals.items() if isinstance(v, torch.Tensor)}
            self.calls.append(([a for a in args if isinstance(a, int) and a > 1 << 20], held))
            return 0
        return call


def _off(*shape):
    """A contiguous tensor that starts where no 16-byte access fits."""
    n = math.prod(shape)
    t = torch.randn(n + 64)[1:1 + n].view(shape)
    assert t.is_contiguous() and t.data_ptr() % 16
    return t


W3, V = (lambda: _off(5, 3)), (lambda: _off(5))
AT_ANY_ADDRESS = {  # the call, and the inputs that 16-byte accesses read
    "conv_fwd": (lambda weight, bias, initial_state: mixer.short_conv_fwd(torch.ones(2, 4, 5), weight, bias, initial_state=initial_state),
                 dict(weight=W3, bias=V, initial_state=lambda: _off(2, 2, 5))),
    "conv_bwd": (lambda d_out, weight, bias, initial_state, d_final_state: mixer.short_conv_bwd(
        torch.ones(2, 4, 5), weight, d_out, bias, initial_state=initial_state, d_final_state=d_final_state),
        dict(d_out=lambda: _off(2, 4, 5), weight=W3, bias=V, initial_state=lambda: _off(2, 2, 5),
             d_final_state=lambda: _off(2, 2, 5))),
    "conv_step": (lambda weight, bias: mixer.short_conv_step(torch.ones(2, 5), torch.ones(2, 2, 5), weight, bias),
                  dict(weight=W3, bias=V)),
    "scan_fwd": (lambda A, D, dt_bias, initial_state: mixer.ssm_scan_fwd(
        torch.ones(2, 4, 5), torch.ones(2, 4, 5), A, torch.ones(2, 4, 1, 8), torch.ones(2, 4, 1, 8), D,
        dt_bias=dt_bias, initial_state=initial_state),
        dict(A=lambda: _off(5, 8), D=V, dt_bias=V, initial_state=lambda: _off(2, 5, 8))),
    "scan_bwd": (lambda A, D, dt_bias, d_out, d_final_state: mixer.ssm_scan_bwd(
        torch.ones(2, 4, 5), torch.ones(2, 4, 5), A, torch.ones(2, 4, 1, 8), torch.ones(2, 4, 1, 8), d_out,
        torch.zeros(256, dtype=torch.uint8), D, dt_bias=dt_bias, d_final_state=d_final_state),
        dict(A=lambda: _off(5, 8), D=V, dt_bias=V, d_out=lambda: _off(2, 4, 5), d_final_state=lambda: _off(2, 5, 8))),
    "scan_step": (lambda A, D, dt_bias: mixer.ssm_scan_step(
        torch.ones(2, 5), torch.ones(2, 5), A, torch.ones(2, 1, 8), torch.ones(2, 1, 8), torch.ones(2, 5, 8), D,
        dt_bias=dt_bias), dict(A=lambda: _off(5, 8), D=V, dt_bias=V)),
    "norm_fwd": (lambda weight, bias: mixer.group_norm_fwd(torch.ones(3, 5), weight, bias), dict(weight=V, bias=V)),
    "norm_bwd": (lambda weight, bias, d_out: mixer.group_norm_bwd(torch.ones(3, 5), d_out, weight, bias),
                 dict(weight=V, bias=V, d_out=lambda: _off(3, 5))),
}


@pytest.mark.parametrize("name", list(AT_ANY_ADDRESS))
def test_inputs_at_any_address(monkeypatch, name):
    """Gradients, states and parameters that are slices of others: the library
    gets their values at a 16-byte boundary."""
    call, inputs = AT_ANY_ADDRESS[name]
    inputs = {k: make() for k, make in inputs.items()}
    lib = Library()
    monkeypatch.setattr(mixer, "load", lambda: lib)
    monkeypatch.setattr(mixer, "_on_gpu", lambda dev, x: None)
    monkeypatch.setattr(mixer, "_current", lambda dev: 0)
    call(**inputs)
    (at, held), = lib.calls
    assert at and not [a for a in at if a % 16]
    for k, t in inputs.items():
        assert held[k].data_ptr() in at and torch.equal(held[k], t), k
    at_16 = {k: t.clone() for k, t in inputs.items()}
    call(**at_16)  # what is aligned is handed on as it is
    assert all(lib.calls[1][1][k] is t for k, t in at_16.items())


def test_a_scan_without_gradients_saves_nothing(monkeypatch):
    """The states for the backward are written only where one can follow."""
    saves = []

    def fwd(u, *args, save_for_backward=False, **kw):
        saves.append(save_for_backward)
        return (u + 0, args[8] if len(args) > 8 else None) + ((u.new_zeros(4),) if save_for_backward else ())

    monkeypatch.setattr(mixer, "ssm_scan_fwd", fwd)
    names = ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "initial_state")
    a = {k: torch.zeros(2) for k in names}
    out, _ = mixer.ssm_scan(**a)
    assert saves == [False] and not out.requires_grad
    for k in names:
        leaf = {**a, k: torch.zeros(2, requires_grad=True)}
        assert mixer.ssm_scan(**leaf)[0].requires_grad and saves[-1], k
        with torch.no_grad():
            assert not mixer.ssm_scan(**leaf)[0].requires_grad and not saves[-1], k


def test_more_groups_than_a_grid_covers_are_refused():
    """Tiny groups in tens of GB: the grid's size, cut to 32 bits, left most of
    the rows alone.  (Without a GPU a call that is not refused ends with 6.)"""
    if torch.cuda.is_available():
        pytest.skip("addresses that are never read, for hosts without a GPU")
    build.build()
    lib, at = gdn.load(), 0x10000
    for channels, groups, limit in ((1, 1, 4 * (2 ** 31 - 1)), (8, 4, 2 ** 31 - 1), (2, 2, 2 ** 32 - 2), (129, 1, 2 ** 31 - 1)):
        for rows, want in ((limit, 6), (limit + 1, 2), (2 ** 34 // groups + 5, 2)):
            x = (at, channels, None, 0, None, None, at, rows, channels, groups, 1e-6, 0, 0, 0, 0)
            assert lib.gdn_norm_fwd(*x, None) == want, (channels, groups, rows)
            bwd = (at, channels, None, 0, None, None, at, at, None, None, None, rows, channels, groups, 1e-6, 0, 0, 0, 0)
            assert lib.gdn_norm_bwd(*bwd, None, 0, None) == want, (channels, groups, rows)


@pytest.mark.parametrize("create_graph", [False, True])
def test_saved_tensors_that_are_recomputed(monkeypatch, create_graph):
    """Under activation checkpointing each saved tensor can be asked for once."""
    f, prefix, fwd, bwd = OPERATORS["norm"]
    monkeypatch.setattr(mixer, prefix + "_fwd", fwd)
    monkeypatch.setattr(mixer, prefix + "_bwd", bwd)
    x, w = torch.randn(2, 5, 4, requires_grad=True), torch.ones(4)
    y = checkpoint(lambda x: f(x, w) * 2, x, use_reentrant=False)
    g, = torch.autograd.grad(y.sum(), x, create_graph=create_graph)
    assert torch.equal(g, 4 * x)
