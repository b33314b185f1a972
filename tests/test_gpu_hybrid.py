"""The layers of examples/hybrid_layers.py: the operators together as they are
used.  Between the operators each tensor is rounded to bf16 (about 1.65e-3 in L2
a time); two paths through two layers differ in some ten of those roundings on
each side, sqrt(20) x 1.65e-3 = 7.4e-3, and gradients pass them twice: 2e-2."""

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
TOL = 2e-2


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_layers.py")
    spec = importlib.util.spec_from_file_location("hybrid_layers", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_steps_continue_packed_prompts(example):
    assert example.continuation_error(example.Hybrid()) <= TOL


def _plain(p, x, layers):
    """The same model in fp64 torch operations on one sequence, (T, width)."""
    rec, win = layers
    T, n = x.shape[0], rec.inner
    u, gate = (x @ p["0.w_in"]).split(n, dim=-1)
    padded = torch.cat([u.new_zeros(rec.taps - 1, n), u])
    u = sum(padded[k:k + T] * p["0.conv_w"][:, k] for k in range(rec.taps)) + p["0.conv_b"]
    r, i = (u @ p["0.w_gates"]).split(n, dim=-1)
    L = -8.0 * torch.nn.functional.softplus(p["0.lam"]) * torch.sigmoid(r)
    a, b = torch.exp(L), torch.sqrt(1 - torch.exp(2 * L)) * torch.sigmoid(i) * u
    h, hs = u.new_zeros(n), []
    for t in range(T):
        h = a[t] * h + b[t]
        hs.append(h)
    x = x + (torch.stack(hs) * torch.nn.functional.silu(gate)) @ p["0.w_out"]
    H, Hk, d = win.H, win.Hk, win.d
    q, k, v = (t.unflatten(-1, (-1, d)) for t in (x @ p["1.w_qkv"]).split([H * d, Hk * d, Hk * d], dim=-1))
    angle = torch.arange(T, device=x.device).double()[:, None, None] * win.inv_freq.double()
    turned = []
    for y, w in ((q, p["1.q_norm"]), (k, p["1.k_norm"])):
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w
        z = torch.complex(*y.chunk(2, -1)) * torch.polar(torch.ones_like(angle), angle)
        turned.append(torch.cat([z.real, z.imag], -1))
    q, k = turned
    ij = torch.arange(T, device=x.device)[:, None] - torch.arange(T, device=x.device)
    see = (ij >= 0) & ((ij < win.window) | (torch.arange(T, device=x.device) < win.sinks))
    s = torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(H // Hk, 1)) / d ** 0.5
    o = torch.einsum("hij,jhd->ihd", torch.softmax(s.masked_fill(~see, float("-inf")), -1), v.repeat_interleave(H // Hk, 1))
    return x + o.flatten(1) @ p["1.w_out"]


@pytest.mark.parametrize("cu", [None, [0, 40, 41, 150]])
def test_outputs_and_gradients_are_the_plain_models(example, cu):
    model = example.Hybrid(seed=4)
    B, T = (1, cu[-1]) if cu else (2, 130)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(B, T, 256, generator=gen, device="cuda").to(torch.bfloat16).requires_grad_()
    g = torch.randn(B, T, 256, generator=gen, device="cuda").to(torch.bfloat16)
    y = model.prompt(x, None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"))
    params = model.parameters()
    grads = torch.autograd.grad(y, [x, *params.values()], g)
    px = x.detach().double().requires_grad_()
    p = {k: v.detach().double().requires_grad_() for k, v in params.items()}
    if cu:
        want = torch.cat([_plain(p, px[0, a:b], model.layers) for a, b in zip(cu[:-1], cu[1:])])[None]
    else:
        want = torch.stack([_plain(p, px[b], model.layers) for b in range(B)])
    ref = torch.autograd.grad(want, [px, *p.values()], g.double())
    for name, got, exact in [("y", y, want)] + list(zip(["x", *params], grads, ref)):
        assert float(((got.double() - exact).norm() / exact.norm()).detach()) <= TOL, name


def test_a_step_in_a_graph(example):
    """One token of every sequence captured once and replayed, the lengths moved on in between."""
    model, rows, more = example.Hybrid(seed=5), 3, 4
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(rows, 60 + more, 256, generator=gen, device="cuda").to(torch.bfloat16)
    slots = torch.arange(rows, dtype=torch.int32, device="cuda")
    prompt = x[:, :60].contiguous()
    want, caches = [], model.cache(rows)
    model.fill(caches, prompt, slots)
    lengths = torch.full((rows,), 60, dtype=torch.int32, device="cuda")
    for s in range(more):
        want.append(model.step(x[:, 60 + s].contiguous(), caches, lengths + s, slots))
    again, token = model.cache(rows), x[:, 60].clone()
    model.step(token, again, lengths, slots)  # the first call of its kind, outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = model.step(token, again, lengths, slots)
    model.fill(again, prompt, slots)
    for s in range(more):
        token.copy_(x[:, 60 + s])
        lengths.fill_(60 + s)
        graph.replay()
        assert float((out.float() - want[s].float()).norm() / want[s].float().norm()) <= TOL, s
