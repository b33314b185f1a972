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
