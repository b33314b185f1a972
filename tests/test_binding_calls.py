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
