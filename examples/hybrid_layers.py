"""Two layers that stand between linear-attention layers, from this package's
operators, for prompts, training and token by token:

- RecurrentLayer: projection -> short convolution -> gated linear recurrence,
  times SiLU of a gate -> projection;
- WindowLayer: one projection for queries, keys and values -> norm and rotation
  of queries and keys -> attention with a sliding window and a few first tokens
  that stay visible -> projection.

Both keep a state of fixed size per sequence, in rows of a cache that a slot
names: the convolution's last inputs and the recurrence's state, or the keys and
values of the window and the first tokens.

Run on a GPU:  python examples/hybrid_layers.py
It reads prompts, continues them token by token from what the prompts left, and
checks that against longer prompts.
"""

from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_sequence_chunked_gb300 import attention, gdn, mixer  # noqa: E402

BF16 = torch.bfloat16


def _linear(gen, n_in, n_out):
    return (torch.randn(n_in, n_out, generator=gen, device="cuda") / math.sqrt(n_in)).to(BF16).requires_grad_()


def _uniform(gen, lo, hi, *shape):
    return (torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo).requires_grad_()


class _Layer:
    def parameters(self):
        return {k: p for k, p in vars(self).items() if isinstance(p, torch.Tensor) and p.requires_grad}


class RecurrentLayer(_Layer):
    def __init__(self, width=256, inner=384, taps=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.inner, self.taps = inner, taps
        self.w_in = _linear(gen, width, 2 * inner)      # input | output gate
        self.w_gates = _linear(gen, inner, 2 * inner)   # gate of the decay | gate of the input
        self.w_out = _linear(gen, inner, width)
        self.conv_w = _uniform(gen, -0.5, 0.5, inner, taps)
        self.conv_b = _uniform(gen, -0.1, 0.1, inner)
        self.lam = _uniform(gen, -6.0, -2.5, inner)

    def _out(self, h, gate):
        return (h * torch.nn.functional.silu(gate)) @ self.w_out

    def prompt(self, x, cu_seqlens=None):
        """x (B, T, width), or packed (1, T, width); returns the output and the
        states after each sequence."""
        u, gate = (x @ self.w_in).split(self.inner, dim=-1)
        u, tail = mixer.short_conv(u, self.conv_w, self.conv_b, activation=None, cu_seqlens=cu_seqlens)
        r, i = (u @ self.w_gates).split(self.inner, dim=-1)   # halves of one projection, read where they are
        h, state = mixer.gated_scan(u, r, i, self.lam, cu_seqlens=cu_seqlens)
        return self._out(h, gate), (tail, state)

    def cache(self, rows):
        return (torch.zeros(rows, self.taps - 1, self.inner, device="cuda", dtype=BF16),
                torch.zeros(rows, self.inner, device="cuda"))

    @torch.no_grad()
    def fill(self, cache, x, slots, cu_seqlens=None):
        y, states = self.prompt(x, cu_seqlens)
        for to, state in zip(cache, states):
            to[slots.long()] = state
        return y

    @torch.no_grad()
    def step(self, x, cache, lengths, slots):
        """x (B, width), one token per row; the cache is updated in place."""
        u, gate = (x @ self.w_in).split(self.inner, dim=-1)
        u = mixer.short_conv_step(u, cache[0], self.conv_w, self.conv_b, activation=None, slots=slots)
        r, i = (u @ self.w_gates).split(self.inner, dim=-1)
        return self._out(mixer.gated_scan_step(u, r, i, self.lam, cache[1], slots=slots), gate)


class WindowLayer(_Layer):
    def __init__(self, width=256, heads=4, key_heads=2, d=64, window=48, sinks=2, base=10000.0, seed=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.Hk, self.d, self.window, self.sinks = heads, key_heads, d, window, sinks
        self.w_qkv = _linear(gen, width, (heads + 2 * key_heads) * d)
        self.w_out = _linear(gen, heads * d, width)
        self.q_norm = _uniform(gen, 0.5, 1.5, d)
        self.k_norm = _uniform(gen, 0.5, 1.5, d)
        self.inv_freq = base ** (-torch.arange(0, d, 2, device="cuda").float() / d)

    def _qkv(self, x, **where):
        """Queries and keys normed and rotated, and the values where the projection left them."""
        qkv = x @ self.w_qkv
        q, k, v = (t.unflatten(-1, (-1, self.d)) for t in qkv.split([self.H * self.d, self.Hk * self.d, self.Hk * self.d], dim=-1))
        q, k = attention.qk_norm_rope(q, k, self.q_norm, self.k_norm, self.inv_freq, **where)
        return q, k, v

    def prompt(self, x, cu_seqlens=None):
        q, k, v = self._qkv(x, cu_seqlens=cu_seqlens)
        o = attention.window_attention(q, k, v, self.window, self.sinks, cu_seqlens=cu_seqlens)
        return o.flatten(-2) @ self.w_out, (k, v)

    def cache(self, rows):
        return tuple(torch.zeros(rows, self.sinks + self.window, self.Hk, self.d, device="cuda", dtype=BF16) for _ in range(2))

    @torch.no_grad()
    def fill(self, cache, x, slots, cu_seqlens=None):
        y, (k, v) = self.prompt(x, cu_seqlens)
        attention.window_cache_fill(k, v, *cache, sinks=self.sinks, cu_seqlens=cu_seqlens, slots=slots)
        return y

    @torch.no_grad()
    def step(self, x, cache, lengths, slots):
        q, k, v = (t[:, 0] for t in self._qkv(x[:, None], positions=lengths[:, None]))
        o = attention.window_attention_step(q, k, v, *cache, lengths, sinks=self.sinks, slots=slots)
        return o.flatten(-2) @ self.w_out


class Hybrid:
    """The two layers in turn, each added to its input."""

    def __init__(self, width=256, seed=0):
        self.layers = [RecurrentLayer(width, seed=seed), WindowLayer(width, seed=seed + 1)]

    def parameters(self):
        return {f"{n}.{k}": p for n, layer in enumerate(self.layers) for k, p in layer.parameters().items()}

    def prompt(self, x, cu_seqlens=None):
        for layer in self.layers:
            x = x + layer.prompt(x, cu_seqlens)[0]
        return x

    def cache(self, rows):
        return [layer.cache(rows) for layer in self.layers]

    @torch.no_grad()
    def fill(self, caches, x, slots, cu_seqlens=None):
        for layer, cache in zip(self.layers, caches):
            x = x + layer.fill(cache, x, slots, cu_seqlens)
        return x

    @torch.no_grad()
    def step(self, x, caches, lengths, slots):
        for layer, cache in zip(self.layers, caches):
            x = x + layer.step(x, cache, lengths, slots)
        return x


def continuation_error(model, lengths=(5, 97, 130), more=6, width=256, seed=2):
    """Relative difference between packed prompts continued token by token, from
    caches in slots, and longer prompts."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    xs = [torch.randn(1, n + more, width, generator=gen, device="cuda").to(BF16) for n in lengths]
    ends = torch.tensor([0, *lengths]).cumsum(0).to(torch.int32).cuda()
    slots = torch.arange(len(lengths), 0, -1, dtype=torch.int32, device="cuda")
    caches = model.cache(len(lengths) + 1)
    model.fill(caches, torch.cat([x[:, :n] for x, n in zip(xs, lengths)], 1), slots, ends)
    at = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    steps = []
    for s in range(more):
        steps.append(model.step(torch.cat([x[:, n + s] for x, n in zip(xs, lengths)]), caches, at + s, slots))
    with torch.no_grad():
        want = torch.stack([model.prompt(x)[0, -more:] for x in xs]).float()
    return float((torch.stack(steps, 1).float() - want).norm() / want.norm())


def main():
    model = Hybrid()
    print(f"prompts continued token by token, relative difference {continuation_error(model):.2e}")
    x = torch.randn(2, 200, 256, device="cuda").to(BF16)
    loss = model.prompt(x).float().square().mean()
    grads = torch.autograd.grad(loss, list(model.parameters().values()))
    print("gradient norms: " + ", ".join(f"{k} {float(g.float().norm()):.3f}" for k, g in zip(model.parameters(), grads)))
    status = gdn.gdn_get_last_device_error()
    assert status == 0, gdn.gdn_status_string(status)


if __name__ == "__main__":
    main()
