"""Paths of the mixer operators beyond the sizes of test_gpu_mixer.py, whose
inputs, comparisons and tolerances these tests use."""

import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import mixer  # noqa: E402

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
