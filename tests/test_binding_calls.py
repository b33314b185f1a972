"""What the binding does around a call, on the CPU: devices, with the CUDA
runtime replaced."""

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
