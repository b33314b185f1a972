"""What the mixer wrappers do around a call, on the CPU: streams, devices,
gradients and addresses, with the kernels and the CUDA runtime replaced."""

import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import mixer  # noqa: E402


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
