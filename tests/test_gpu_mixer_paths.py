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
