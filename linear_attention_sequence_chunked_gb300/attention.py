"""The operators of the attention layers that a linear-attention model puts
between its others: the norm and rotation of queries and keys.

As in mixer.py, nothing is computed here: arguments are checked and handed to
the CUDA kernels of ``_build/libgdn.so`` (include/gdn.h has the formulas and
layouts), without a CPU fallback.  ``*_fwd`` / ``*_bwd`` are the explicit forms
and take `stream=`, in place of the current stream; the others are the same
behind torch.autograd (first derivatives only).  All tensors are on the current
device.
"""

from __future__ import annotations

import torch

from ._first_order import first_order
from .gdn import _check, _on_stream, _workspace, load
from .mixer import _aligned, _current, _dense, _dtype, _is, _on_gpu, _out, _rows, _sequences

HEAD_SIZES = (32, 64, 128, 256)


# ----------------------------------------------------------------------------
# norm and rotation of queries and keys
# ----------------------------------------------------------------------------

def _rope_args(q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, interleaved, eps):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"q and k must be (B, T, heads, d), got shapes {tuple(q.shape)} and {tuple(k.shape)}")
    dtype, dev = _dtype(q, "q"), q.get_device()
    B, T, H, d = q.shape
    Hk = k.shape[2]
    _is("k", k, (B, T, Hk, d), q.dtype, dev)
    if d not in HEAD_SIZES:
        raise ValueError(f"the head size must be one of {HEAD_SIZES}, got {d}")
    pairs = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1 or inv_freq.numel() % 4 or 2 * inv_freq.numel() > d:
            raise ValueError(f"inv_freq must hold a multiple of 4 frequencies, at most {d // 2}, "
                             f"got shape {tuple(inv_freq.shape)}")
        pairs = inv_freq.numel()
    n, cu = _sequences(q, cu_seqlens, dev, "q")
    args = (*_rows(q, H * d, 2), *_rows(k, Hk * d, 2), _dense("q_weight", q_weight, (d,), torch.float32, dev),
            _dense("k_weight", k_weight, (d,), torch.float32, dev),
            _dense("inv_freq", inv_freq, (pairs,), torch.float32, dev),
            _dense("positions", positions, (B, T), torch.int32, dev), cu)
    _on_gpu(dev, q)
    return dev, args, (n, T, H, Hk, d, pairs, int(interleaved), eps, dtype)


def qk_norm_rope_fwd(q, k, q_weight=None, k_weight=None, inv_freq=None, positions=None, cu_seqlens=None, eps=1e-6,
                     interleaved=False, stream=None):
    """RMS norm of every head of q (B, T, H, d) and k (B, T, Hk, d), times its
    weight (d), and the rotation by the token's position: pair j of channels
    (j and j + n of n = len(inv_freq); 2j and 2j + 1 with interleaved) turns by
    position x inv_freq[j] radians, channels from 2n on stay.  positions (B, T)
    int32; by default a token's place in its sequence.  q and k may be slices of
    one projection.  Returns (q, k), dense."""
    if stream is not None:
        return _on_stream(qk_norm_rope_fwd, locals())
    q_weight, k_weight, inv_freq = _aligned(q_weight, k_weight, inv_freq)
    dev, args, dims = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, interleaved, eps)
    qo, ko = q.new_empty(q.shape), k.new_empty(k.shape)
    _check(load().gdn_rope_fwd(*args, qo.data_ptr(), ko.data_ptr(), *dims, _current(dev)), "gdn_rope_fwd")
    return qo, ko


def qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight=None, k_weight=None, inv_freq=None, positions=None,
                     cu_seqlens=None, eps=1e-6, interleaved=False, stream=None):
    """Gradients of qk_norm_rope_fwd from its inputs and the gradients of its
    outputs: a dict of dq, dk, and dq_weight and dk_weight for those that were
    given."""
    if stream is not None:
        return _on_stream(qk_norm_rope_bwd, locals())
    q_weight, k_weight, inv_freq, dq_out, dk_out = _aligned(q_weight, k_weight, inv_freq, dq_out, dk_out)
    dev, args, dims = _rope_args(q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, interleaved, eps)
    gq = _dense("dq_out", dq_out, q.shape, q.dtype, dev)
    gk = _dense("dk_out", dk_out, k.shape, k.dtype, dev)
    res = {"dq": q.new_empty(q.shape), "dk": k.new_empty(k.shape)}
    if q_weight is not None:
        res["dq_weight"] = torch.empty_like(q_weight)
    if k_weight is not None:
        res["dk_weight"] = torch.empty_like(k_weight)
    lib = load()
    nbytes = 0
    if len(res) > 2:
        nbytes = lib.gdn_rope_bwd_workspace_size(*dims[:5], int(cu_seqlens is not None))
    ws = _workspace(nbytes, q.device)
    _check(lib.gdn_rope_bwd(*args, gq, gk, res["dq"].data_ptr(), res["dk"].data_ptr(), _out(res, "dq_weight"),
                            _out(res, "dk_weight"), *dims, None if ws is None else ws.data_ptr(), nbytes,
                            _current(dev)), "gdn_rope_bwd")
    return res


# ----------------------------------------------------------------------------
# autograd
# ----------------------------------------------------------------------------

_FUNCTIONS = {}


def _functions():
    if _FUNCTIONS:
        return _FUNCTIONS

    def dense(g, like):
        return like.new_zeros(like.shape) if g is None else g.to(like.dtype).contiguous()

    class QkNormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, eps, interleaved):
            ctx.save_for_backward(q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens)
            ctx.rest = (eps, interleaved)
            ctx.set_materialize_grads(False)
            return qk_norm_rope_fwd(q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, *ctx.rest)

        @staticmethod
        @first_order
        def backward(ctx, saved_tensors, dq_out, dk_out):
            q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens = saved_tensors
            r = qk_norm_rope_bwd(q, k, dense(dq_out, q), dense(dk_out, k), q_weight, k_weight, inv_freq, positions,
                                 cu_seqlens, *ctx.rest)
            return (r["dq"], r["dk"], r.get("dq_weight"), r.get("dk_weight")) + (None,) * 5

    _FUNCTIONS.update(rope=QkNormRope)
    return _FUNCTIONS


def qk_norm_rope(q, k, q_weight=None, k_weight=None, inv_freq=None, positions=None, cu_seqlens=None, eps=1e-6,
                 interleaved=False):
    """qk_norm_rope_fwd with autograd (q, k, q_weight, k_weight; the frequencies
    are constants).  Returns (q, k)."""
    if inv_freq is not None and inv_freq.requires_grad:
        raise ValueError("inv_freq has no gradient here: pass it detached")
    return _functions()["rope"].apply(q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, eps, interleaved)
