"""What the binding does around a call, on the CPU: devices, with the CUDA
runtime replaced."""

import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import gdn  # noqa: E402


def _tensor(index, address=0x10000):
    return types.SimpleNamespace(is_contiguous=lambda: True, device=torch.device("cuda", index),
                                 get_device=lambda: index, data_ptr=lambda: address)


def test_a_tensor_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(gdn, "_device", lambda: 0, raising=False)
    assert gdn._ptr(_tensor(0)) == 0x10000
    with pytest.raises(ValueError, match="on cuda:1, the current device is cuda:0"):
        gdn._ptr(_tensor(1))


def test_second_derivatives_are_refused(monkeypatch):
    """With 2 q d_out and the like in the kernels' place: where another path to
    the same input has a second derivative, only that one would come back."""
    def fwd(q, k, v, g, beta, initial_state=None, **kw):
        return q * q, initial_state, torch.zeros(4, dtype=torch.uint8)

    def bwd(q, k, v, g, beta, d_out, **kw):
        return dict(dq=2 * q * d_out, dk=0 * k, dv=0 * v, dg=0 * g, dbeta=0 * beta, d_initial_state=None)

    monkeypatch.setattr(gdn, "chunk_gated_delta_rule_fwd", fwd)
    monkeypatch.setattr(gdn, "chunk_gated_delta_rule_bwd", bwd)
    x = torch.randn(1, 4, 2, 8).bfloat16().requires_grad_()
    g, beta, h = torch.zeros(1, 4, 2), torch.zeros(1, 4, 2).bfloat16(), torch.zeros(1, 2, 8, 8)

    def f():
        return gdn.chunk_gated_delta_rule(x, x.detach(), x.detach(), g, beta, initial_state=h)[0].sum()

    dx, = torch.autograd.grad(f(), x, create_graph=True)
    assert torch.equal(dx, 2 * x)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        (dx.sum() + (x ** 3).sum()).backward()
    f().backward()
    assert torch.equal(x.grad, 2 * x)


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is a CUDA one."""
    is_cuda = property(lambda self: True)


CALLS = {  # the wrapper, its further arguments, and the library call in it
    "chunk_gated_delta_rule_fwd": ("g", {}, "gdn_chunk_fwd"),
    "chunk_gated_delta_rule_fwd (saving)": ("g", dict(save_for_backward=True), "gdn_chunk_fwd_save"),
    "chunk_gated_delta_rule_fwd_split": ("g", dict(nseg=2), "gdn_chunk_fwd_split"),
    "chunk_gated_delta_rule_bwd": ("g", dict(d_out="v"), "gdn_chunk_bwd"),
    "chunk_gated_delta_rule_bwd (saved)": ("g", dict(d_out="v", saved="saved"), "gdn_chunk_bwd_saved"),
    "chunk_kda_fwd": ("gk", {}, "gdn_kda_chunk_fwd"),
    "chunk_kda_bwd": ("gk", dict(d_out="v"), "gdn_kda_chunk_bwd"),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_memory_of_a_call_on_another_stream(monkeypatch, name):
    """Outputs and workspaces come from the given stream's memory (a workspace
    is given back when the call returns), inputs stay until it is through with
    them, outputs until the caller's stream is."""
    gate, more, inner = CALLS[name]
    bf = torch.bfloat16
    t = dict(q=torch.zeros(1, 64, 2, 64, dtype=bf), v=torch.zeros(1, 64, 2, 64, dtype=bf), g=torch.zeros(1, 64, 2),
             gk=torch.zeros(1, 64, 2, 64), beta=torch.zeros(1, 64, 2, dtype=bf), saved=torch.zeros(64, dtype=torch.uint8))
    t = {k: v.as_subclass(OnGpu) for k, v in t.items()}
    stream = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=77)
    now, recorded, made, empty = ["caller"], [], [], torch.empty

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        yield
        now.pop()

    def take(*a, **k):
        x = empty(*a, **k)
        made.append((x, now[-1]))
        return x

    def record(x, s):
        recorded.append((x, s))

    def library(*args, **kw):
        assert now[-1] is stream and (args[-1] is None or not hasattr(args[-1], "cuda_stream"))
        assert all(any(x is t[k] and s is stream for x, s in recorded) for k in ("q", "v", gate, "beta"))

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "caller")
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    monkeypatch.setattr(torch, "empty", take)
    monkeypatch.setattr(gdn, "load", lambda: types.SimpleNamespace(**{f: lambda *a: 256 for f in SIZES}))
    monkeypatch.setattr(gdn, inner, library)
    more = {k: t.get(v, v) if isinstance(v, str) else v for k, v in more.items()}
    out = getattr(gdn, name.split()[0])(t["q"], t["q"], t["v"], t[gate], t["beta"], stream=stream, **more)
    out = list(out.values()) if isinstance(out, dict) else list(out)
    assert made and all(s is stream for _, s in made)
    assert all(any(x is o and s == "caller" for x, s in recorded) for o in out)
    assert now == ["caller"]


SIZES = ("gdn_chunk_fwd_workspace_size", "gdn_chunk_bwd_workspace_size", "gdn_chunk_saved_size",
         "gdn_chunk_bwd_saved_workspace_size", "gdn_chunk_fwd_split_workspace_size", "gdn_kda_chunk_fwd_workspace_size",
         "gdn_kda_chunk_bwd_workspace_size")
