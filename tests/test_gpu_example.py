"""The mixer layers of examples/mixer_layers.py: a prompt continued token by
token equals one longer prompt up to the bf16 roundings between the operators
(each about 2e-3 in L2, five or six of them on different paths: 2e-2 bounds
them), and gradient descent lowers the loss."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixer_layers.py")
    spec = importlib.util.spec_from_file_location("mixer_layers", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("name", ["SsmMixer", "DeltaMixer"])
def test_decode_continues_the_prompt(example, name):
    assert example.continuation_error(getattr(example, name)()) <= 2e-2


def test_training_lowers_the_loss(example):
    losses = example.train(example.SsmMixer())
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_packed_prompt_equals_separate_ones(example):
    layer = example.SsmMixer()
    x = torch.randn(1, 150, 512, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 70, 71, 150], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        y, (conv, state) = layer.prompt(x, cu)
        for n, (a, b) in enumerate(((0, 70), (70, 71), (71, 150))):
            y1, (c1, s1) = layer.prompt(x[:, a:b].contiguous())
            # the projections may take another library kernel at another size
            assert float((y1.float() - y[:, a:b].float()).norm() / y1.float().norm()) <= 2e-2
            assert float((s1[0] - state[n]).norm() / s1.norm()) <= 2e-2
