"""Backwards that end at the first derivative."""

from __future__ import annotations

import functools

import torch


class _Final(torch.autograd.Function):
    """Gradients that cannot be differentiated again, and what they depend on."""

    @staticmethod
    def forward(ctx, count, *tensors):
        return tensors[:count]

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the gradients of this operator cannot be differentiated again")


def first_order(backward):
    """backward(ctx, saved tensors, *grads) as an autograd Function's backward,
    for gradients that come from kernels and carry no graph.  Where one is asked
    for (create_graph), differentiating them raises: as constants they would
    silently drop out of a second derivative."""
    @functools.wraps(backward)
    def wrapped(ctx, *grads):
        saved = ctx.saved_tensors  # once: hooks that recompute them refuse a second time
        with torch.no_grad():
            out = backward(ctx, saved, *grads)
        if not torch.is_grad_enabled():
            return out
        made = [g for g in out if g is not None]
        final = iter(_Final.apply(len(made), *made, *saved, *grads))
        return tuple(None if g is None else next(final) for g in out)
    return wrapped
