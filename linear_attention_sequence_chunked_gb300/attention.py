"""The operators of the attention layers that a linear-attention model puts
between its others: the norm and rotation of queries and keys, and attention
with a sliding window and first tokens that stay visible, for prompts, for
training, and token by token on a cache of fixed size.

As in mixer.py, nothing is computed here: arguments are checked and handed to
the CUDA kernels of ``_build/libgdn.so`` (include/gdn.h has the formulas and
layouts), without a CPU fallback.  ``*_fwd`` / ``*_bwd`` are the explicit forms
and take `stream=`, in place of the current stream; the others are the same
behind torch.autograd (first derivatives in reverse mode only).  All tensors are
on the current device.
"""

from __future__ import annotations

import torch

from ._first_order import first_order
from .gdn import _check, _on_stream, _workspace, load
from .mixer import _aligned, _current, _dense, _differentiated, _dtype, _is, _new, _on_gpu, _out, _rows, _sequences

_BF16 = torch.bfloat16
HEAD_SIZES = (32, 64, 128, 256)
WINDOW_HEAD_SIZES = (64, 128)
MAX_SINKS = 128


# ----------------------------------------------------------------------------
# norm and rotation of queries and keys
# ----------------------------------------------------------------------------

def _rope_args(q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, interleaved, eps):
    qs, ks = q.shape, k.shape
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError(f"q and k must be (B, T, heads, d), got shapes {tuple(qs)} and {tuple(ks)}")
    dtype, dev = _dtype(q, "q"), q.get_device()
    B, T, H, d = qs
    Hk = ks[2]
    _is("k", k, (B, T, Hk, d), q.dtype, dev)
    if d not in HEAD_SIZES:
        raise ValueError(f"the head size must be one of {HEAD_SIZES}, got {d}")
    pairs = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1 or inv_freq.shape[0] % 4 or 2 * inv_freq.shape[0] > d:
            raise ValueError(f"inv_freq must hold a multiple of 4 frequencies, at most {d // 2}, "
                             f"got shape {tuple(inv_freq.shape)}")
        pairs = inv_freq.shape[0]
    n, cu = (B, None) if cu_seqlens is None else _sequences(q, cu_seqlens, dev, "q")
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
    qo, ko = _new(q), _new(k)
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
    res = {"dq": _new(q), "dk": _new(k)}
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
# attention with a sliding window and first tokens that stay visible
# ----------------------------------------------------------------------------

def _pieces(x, width, held):
    """(address, row stride) of rows of heads that the kernels copy in 16-byte
    pieces; of a copy, which the caller holds until its launch, where they lie
    elsewhere."""
    at, stride = (x.data_ptr(), width) if x.is_contiguous() else _rows(x, width, 2)
    if at & 15 or stride & 7:
        held.append(x.clone(memory_format=torch.contiguous_format))
        at, stride = held[-1].data_ptr(), width
    return at, stride


def _window_args(q, k, v, window, sinks, scale, dims):
    """Checks shared by the attention and its step (q of 4 or 3 dimensions).
    The copies of the answer are held until the launch."""
    shape, kv, dev = q.shape, k.shape, q.get_device()
    if len(shape) != dims or len(kv) != dims:
        raise ValueError(f"q and k must be {'(B, T, heads, d)' if dims == 4 else '(B, heads, d)'}, "
                         f"got shapes {tuple(shape)} and {tuple(kv)}")
    if q.dtype is not _BF16:
        raise ValueError(f"q must be {_BF16}, got {q.dtype}")
    H, d = shape[-2:]
    Hk = kv[-2]
    if kv[-1] != d or kv[0] != shape[0] or kv[1] != (shape[1] if dims == 4 else Hk) or k.dtype is not _BF16 or k.get_device() != dev:
        _is("k", k, shape[:-2] + (Hk, d), _BF16, dev)
    if v.shape != kv or v.dtype is not _BF16 or v.get_device() != dev:
        _is("v", v, kv, _BF16, dev)
    if d not in WINDOW_HEAD_SIZES:
        raise ValueError(f"the head size must be one of {WINDOW_HEAD_SIZES}, got {d}")
    if Hk < 1 or H % Hk or H < 1:
        raise ValueError(f"the {H} query heads must divide into the {Hk} key heads")
    _window_sizes(window, sinks)
    scale = d ** -0.5 if scale is None else float(scale)
    if not 0 < scale < 3e38:
        raise ValueError(f"scale must be positive and finite, got {scale}")
    _on_gpu(dev, q)
    held = []
    return dev, held, (*_pieces(q, H * d, held), *_pieces(k, Hk * d, held), *_pieces(v, Hk * d, held)), H, Hk, d, scale


def _window_sizes(window, sinks):
    if window < 1:
        raise ValueError(f"window must be at least 1 (a token sees itself), got {window}")
    if not 0 <= sinks <= MAX_SINKS:
        raise ValueError(f"sinks must be in 0 .. {MAX_SINKS}, got {sinks}")


def window_attention_fwd(q, k, v, window, sinks=0, scale=None, cu_seqlens=None, save_for_backward=False, stream=None):
    """Causal attention in which token i sees j <= i with i - j < window or
    j < sinks: q (B, T, H, d), k and v (B, T, Hk, d) bf16, H a multiple of Hk
    (query head h reads key head h // (H // Hk)), scale by default d^-1/2.  All
    three may be slices of one projection.  Returns out (B, T, H, d), or (out,
    lse) with save_for_backward: lse (B, H, T) fp32, the log of each row's sum."""
    if stream is not None:
        return _on_stream(window_attention_fwd, locals())
    dev, held, args, H, Hk, d, scale = _window_args(q, k, v, window, sinks, scale, 4)
    n, cu = _sequences(q, cu_seqlens, dev, "q")
    B, T = q.shape[:2]
    out = _new(q)
    lse = torch.empty((B, H, T), dtype=torch.float32, device=q.device) if save_for_backward else None
    _check(load().gdn_window_fwd(*args, cu, out.data_ptr(), None if lse is None else lse.data_ptr(), n, T, H, Hk, d,
                                 min(window, max(T, 1)), sinks, scale, _current(dev)), "gdn_window_fwd")
    return (out, lse) if save_for_backward else out


def window_attention_bwd(q, k, v, out, lse, d_out, window, sinks=0, scale=None, cu_seqlens=None, stream=None):
    """Gradients of window_attention_fwd from its inputs and the (out, lse) that
    it returned: a dict of dq, dk and dv."""
    if stream is not None:
        return _on_stream(window_attention_bwd, locals())
    out, lse, d_out = _aligned(out, lse, d_out)
    dev, held, args, H, Hk, d, scale = _window_args(q, k, v, window, sinks, scale, 4)
    n, cu = _sequences(q, cu_seqlens, dev, "q")
    B, T = q.shape[:2]
    o = _dense("out", out, q.shape, q.dtype, dev)
    s = _dense("lse", lse, (B, H, T), torch.float32, dev)
    g = _dense("d_out", d_out, q.shape, q.dtype, dev)
    res = {"dq": _new(q), "dk": _new(k), "dv": _new(v)}
    window = min(window, max(T, 1))
    lib = load()
    nbytes = lib.gdn_window_bwd_workspace_size(n, T, H, Hk, d, window, sinks, int(cu_seqlens is not None))
    ws = _workspace(nbytes, q.device)
    _check(lib.gdn_window_bwd(*args, cu, o, s, g, res["dq"].data_ptr(), res["dk"].data_ptr(), res["dv"].data_ptr(), n, T,
                              H, Hk, d, window, sinks, scale, None if ws is None else ws.data_ptr(), nbytes,
                              _current(dev)), "gdn_window_bwd")
    return res


def _caches(k_cache, v_cache, Hk, d, sinks, dev):
    """Addresses of the two caches, and how many there are of how many rows."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[1] <= sinks or v_cache.shape != shape:
        raise ValueError(f"the caches must be (S, sinks + window, {Hk}, {d}) alike, got shapes {tuple(shape)} and "
                         f"{tuple(v_cache.shape)}")
    S, rows = shape[:2]
    kc = _dense("k_cache", k_cache, (S, rows, Hk, d), _BF16, dev)
    vc = _dense("v_cache", v_cache, (S, rows, Hk, d), _BF16, dev)
    if (kc | vc) & 15:
        raise ValueError("the caches must start at 16-byte boundaries: they are updated in place")
    return kc, vc, S, rows


def window_attention_step(q, k, v, k_cache, v_cache, lengths, sinks=0, scale=None, slots=None, stream=None):
    """One token per row: q (B, H, d), k and v (B, Hk, d), and caches (S, sinks +
    window, Hk, d) that hold token p in row p, from p = sinks on in row sinks +
    (p - sinks) % window.  lengths (B, int32): the tokens that each row's sequence
    has behind it, so the position of this one, whose key and value are written
    into the caches (lengths stays; negative: an idle row, whose output is zero).
    slots as in mixer.short_conv_step.  Returns out (B, H, d)."""
    if stream is not None:
        return _on_stream(window_attention_step, locals())
    dev, held, args, H, Hk, d, scale = _window_args(q, k, v, 1, sinks, scale, 3)
    B = q.shape[0]
    kc, vc, S, rows = _caches(k_cache, v_cache, Hk, d, sinks, dev)
    if slots is None and S < B:
        raise ValueError(f"the caches hold {S} rows for a batch of {B}")
    ln = _dense("lengths", lengths, (B,), torch.int32, dev)
    sl = _dense("slots", slots, (B,), torch.int32, dev)
    out = _new(q)
    _check(load().gdn_window_step(*args, kc, vc, ln, sl, out.data_ptr(), B, S, H, Hk, d, rows - sinks, sinks, scale,
                                  _current(dev)), "gdn_window_step")
    return out


def window_cache_fill(k, v, k_cache, v_cache, sinks=0, cu_seqlens=None, slots=None, stream=None):
    """Puts what the next token of each prompt looks at into its cache (laid out
    as in window_attention_step): k, v (B, T, Hk, d), slots (one per sequence,
    int32; negative: none).  Rows that hold no token keep what they have."""
    if stream is not None:
        return _on_stream(window_cache_fill, locals())
    if k.dim() != 4:
        raise ValueError(f"k must be (B, T, heads, d), got shape {tuple(k.shape)}")
    dev, held, args, _, Hk, d, _ = _window_args(k, k, v, 1, sinks, None, 4)
    n, cu = _sequences(k, cu_seqlens, dev, "k")
    kc, vc, S, rows = _caches(k_cache, v_cache, Hk, d, sinks, dev)
    if slots is None and S < n:
        raise ValueError(f"the caches hold {S} rows for {n} sequences")
    sl = _dense("slots", slots, (n,), torch.int32, dev)
    _check(load().gdn_window_fill(*args[2:], cu, sl, kc, vc, n, k.shape[1], S, Hk, d, rows - sinks, sinks,
                                  _current(dev)), "gdn_window_fill")


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

    class WindowAttention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, window, sinks, scale, cu_seqlens):
            out, lse = window_attention_fwd(q, k, v, window, sinks, scale, cu_seqlens, save_for_backward=True)
            ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
            ctx.rest = (window, sinks, scale)
            return out

        @staticmethod
        @first_order
        def backward(ctx, saved_tensors, d_out):
            q, k, v, out, lse, cu_seqlens = saved_tensors
            r = window_attention_bwd(q, k, v, out, lse, dense(d_out, q), *ctx.rest, cu_seqlens)
            return (r["dq"], r["dk"], r["dv"]) + (None,) * 4

    _FUNCTIONS.update(rope=QkNormRope, window=WindowAttention)
    return _FUNCTIONS


def qk_norm_rope(q, k, q_weight=None, k_weight=None, inv_freq=None, positions=None, cu_seqlens=None, eps=1e-6,
                 interleaved=False):
    """qk_norm_rope_fwd with autograd (q, k, q_weight, k_weight; the frequencies
    are constants).  Returns (q, k)."""
    if inv_freq is not None and inv_freq.requires_grad:
        raise ValueError("inv_freq has no gradient here: pass it detached")
    return _functions()["rope"].apply(q, k, q_weight, k_weight, inv_freq, positions, cu_seqlens, eps, interleaved)


def window_attention(q, k, v, window, sinks=0, scale=None, cu_seqlens=None):
    """window_attention_fwd with autograd (q, k, v).  The rows' sums are kept
    where a backward can follow."""
    if not _differentiated(q, k, v):
        return window_attention_fwd(q, k, v, window, sinks, scale, cu_seqlens)
    return _functions()["window"].apply(q, k, v, window, sinks, scale, cu_seqlens)
