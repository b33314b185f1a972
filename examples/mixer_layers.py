"""Two mixer layers from this package's operators, for prompts, training and
token by token:

- SsmMixer: projection -> short convolution + SiLU -> selective state space
  scan -> group norm gated by SiLU -> projection;
- DeltaMixer: projections -> short convolution + SiLU on q, k and v together ->
  prologue (q/k norm, gates) -> gated delta rule -> norm per head gated by
  SiLU -> projection ("Research Sprint Day 2 - Rooflines", GDN layer pseudocode).

Run on a GPU:  python examples/mixer_layers.py
It reads a prompt, continues it token by token from the states that the prompt
left, checks that against one longer prompt, and takes a few training steps.
"""

from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_sequence_chunked_gb300 import gdn, mixer  # noqa: E402

BF16 = torch.bfloat16


def _linear(gen, n_in, n_out):
    w = torch.randn(n_in, n_out, generator=gen, device="cuda") / math.sqrt(n_in)
    return w.to(BF16).requires_grad_()


def _uniform(gen, lo, hi, *shape):
    return (torch.rand(*shape, generator=gen, device="cuda") * (hi - lo) + lo).requires_grad_()


class SsmMixer:
    def __init__(self, width=512, inner=1024, states=16, norm_groups=8, taps=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.inner, self.states, self.groups, self.taps = inner, states, norm_groups, taps
        self.rank = inner // 16
        self.w_in = _linear(gen, width, 2 * inner)                    # u | gate
        self.w_x = _linear(gen, inner, self.rank + 2 * states)        # step rank | B | C
        self.w_dt = _linear(gen, self.rank, inner)
        self.w_out = _linear(gen, inner, width)
        self.conv_w = _uniform(gen, -0.5, 0.5, inner, taps)
        self.conv_b = _uniform(gen, -0.1, 0.1, inner)
        self.A_log = torch.log(torch.arange(1, states + 1, device="cuda").float()).repeat(inner, 1).requires_grad_()
        self.D = torch.ones(inner, device="cuda", requires_grad=True)
        self.dt_bias = _uniform(gen, -5.0, -2.0, inner)
        self.norm_w = torch.ones(inner, device="cuda", requires_grad=True)

    def parameters(self):
        return [p for p in vars(self).values() if isinstance(p, torch.Tensor)]

    def _bc(self, u):
        """The step and B, C of the scan, all slices of one projection of u."""
        x = u @ self.w_x
        r, n = self.rank, self.states
        return x[..., :r] @ self.w_dt, x[..., r:r + n].unflatten(-1, (1, n)), x[..., r + n:].unflatten(-1, (1, n))

    def _out(self, y, gate):
        y = mixer.group_norm(y, self.norm_w, gate=gate, groups=self.groups, gate_first=True)
        return y @ self.w_out

    def prompt(self, x, cu_seqlens=None):
        """x (B, T, width), or packed (1, T, width); returns the output and the
        state that the next token starts from."""
        xz = x @ self.w_in
        u, gate = xz[..., :self.inner], xz[..., self.inner:]          # strided halves, read as they are
        u, conv_state = mixer.short_conv(u, self.conv_w, self.conv_b, cu_seqlens=cu_seqlens)
        dt, B, C = self._bc(u)
        y, state = mixer.ssm_scan(u, dt, -torch.exp(self.A_log), B, C, D=self.D, dt_bias=self.dt_bias,
                                  cu_seqlens=cu_seqlens)
        return self._out(y, gate), (conv_state, state)

    @torch.no_grad()
    def step(self, x, cache, slots=None):
        """x (B, width), one token per row; the cache is updated in place."""
        conv_state, state = cache
        xz = x @ self.w_in
        u = mixer.short_conv_step(xz[:, :self.inner], conv_state, self.conv_w, self.conv_b, slots=slots)
        dt, B, C = self._bc(u)
        y = mixer.ssm_scan_step(u, dt, -torch.exp(self.A_log), B, C, state, D=self.D, dt_bias=self.dt_bias, slots=slots)
        return self._out(y, xz[:, self.inner:])


class DeltaMixer:
    """Inference only: the prologue's backward is called explicitly elsewhere."""

    def __init__(self, width=512, heads=4, d_k=64, d_v=128, taps=4, seed=1):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.d_k, self.d_v = heads, d_k, d_v
        self.sizes = [heads * d_k, heads * d_k, heads * d_v]
        self.w_qkv = _linear(gen, width, sum(self.sizes)).detach()
        self.w_gates = _linear(gen, width, 2 * heads).detach()
        self.w_z = _linear(gen, width, heads * d_v).detach()
        self.w_out = _linear(gen, heads * d_v, width).detach()
        self.conv_w = _uniform(gen, -0.5, 0.5, sum(self.sizes), taps).detach()
        self.A_log = _uniform(gen, 0.0, 1.0, heads).detach()
        self.dt_bias = _uniform(gen, -3.0, -1.0, heads).detach()
        self.norm_w = torch.ones(d_v, device="cuda")

    def _heads(self, x, qkv):
        """The delta rule's inputs from rows of x and of the convolved projection."""
        rows = x.shape[0]
        q, k, v = (t.contiguous().view(rows, self.H, -1) for t in qkv.split(self.sizes, dim=-1))
        a, b = (t.float().contiguous() for t in (x @ self.w_gates).chunk(2, dim=-1))
        qn, kn = torch.empty_like(q), torch.empty_like(k)
        g = torch.empty(rows, self.H, device="cuda")
        beta = torch.empty(rows, self.H, device="cuda", dtype=BF16)
        gdn.gdn_prologue_fwd(q, k, a, b, self.A_log, self.dt_bias, 1, 0.0, 1.0, qn, kn, g, beta, rows, self.H, self.d_k)
        return qn, kn, v, g, beta

    def _out(self, o, x):
        gate = (x @ self.w_z).view(-1, self.d_v)
        y = mixer.group_norm_fwd(o.view(-1, self.d_v), self.norm_w, gate=gate)   # one norm weight for all heads
        return y.view(x.shape[0], -1) @ self.w_out

    @torch.no_grad()
    def prompt(self, x):
        B, T, _ = x.shape
        qkv, conv_state = mixer.short_conv_fwd(x @ self.w_qkv, self.conv_w, output_final_state=True)
        flat = x.reshape(B * T, -1)
        ins = [t.view(B, T, *t.shape[1:]) for t in self._heads(flat, qkv.view(B * T, -1))]
        o, state = gdn.chunk_gated_delta_rule_fwd(*ins)
        return self._out(o, flat).view(B, T, -1), (conv_state, state)

    @torch.no_grad()
    def step(self, x, cache):
        conv_state, state = cache
        B = x.shape[0]
        qkv = mixer.short_conv_step(x @ self.w_qkv, conv_state, self.conv_w)
        q, k, v, g, beta = self._heads(x, qkv)
        o, new = torch.empty_like(v), torch.empty_like(state)
        gdn.gdn_recurrent_fwd(q, k, v, g, beta, self.d_k ** -0.5, state, None, o, new, B, 1, self.H, self.d_k, self.d_v)
        state.copy_(new)
        return self._out(o, x)


def continuation_error(layer, B=3, T=97, more=6, width=512, seed=2):
    """Relative difference between a prompt continued token by token and one longer prompt."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, T + more, width, generator=gen, device="cuda").to(BF16)
    with torch.no_grad():
        whole, _ = layer.prompt(x)
        _, cache = layer.prompt(x[:, :T].contiguous())
        steps = torch.stack([layer.step(x[:, t].contiguous(), cache) for t in range(T, T + more)], 1)
    want = whole[:, T:].float()
    return float((steps.float() - want).norm() / want.norm())


def train(layer, steps=5, B=2, T=160, width=512, lr=0.2, seed=3):
    """Plain gradient descent on a fixed batch; returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, T, width, generator=gen, device="cuda").to(BF16)
    target = torch.randn(B, T, width, generator=gen, device="cuda")
    losses = []
    for _ in range(steps):
        y, _ = layer.prompt(x)
        loss = (y.float() - target).square().mean()
        grads = torch.autograd.grad(loss, layer.parameters())
        with torch.no_grad():
            for p, g in zip(layer.parameters(), grads):
                p -= lr * g.to(p.dtype)
        losses.append(float(loss.detach()))
    return losses


def main():
    ssm, delta = SsmMixer(), DeltaMixer()
    print(f"state space mixer: prompt continued token by token, relative difference {continuation_error(ssm):.2e}")
    print(f"delta rule mixer:  prompt continued token by token, relative difference {continuation_error(delta):.2e}")
    print("state space mixer: losses " + " ".join(f"{v:.4f}" for v in train(ssm)))
    status = gdn.gdn_get_last_device_error()
    assert status == 0, gdn.gdn_status_string(status)


if __name__ == "__main__":
    main()
