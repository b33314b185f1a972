"""The operators around the recurrence of a mixer layer: a short causal
convolution, the selective state space scan, and the group norm with an
activation; for prompts, for training, and token by token.

As in gdn.py, nothing is computed here: arguments are checked and handed to
the CUDA kernels of ``_build/libgdn.so`` (include/gdn.h has the formulas and
layouts), without a CPU fallback.  ``*_fwd`` / ``*_bwd`` / ``*_step`` allocate
their outputs and workspaces with torch; short_conv, ssm_scan and group_norm
are the same forwards and backwards behind torch.autograd (first derivatives
only: a second one raises).  The former also
take `stream=`, in place of the current stream; as with any stream, the caller
has it wait for what produces the inputs.  All tensors are on the current device.

Activations are channels last and bf16 or fp32, one type per call; parameters
and the states of the scan are fp32.  The activation inputs x, gate, u, dt, z,
B and C may be slices of a wider projection: any tensor whose rows are dense
and evenly spaced.  Other inputs are contiguous, and copied where they do not
start at a 16-byte boundary; a state cache that a step updates does.
"""

from __future__ import annotations

import torch

from ._first_order import first_order
from .gdn import _check, _on_stream, _workspace, load

_ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "sigmoid": 2}
STATE_SIZES = (8, 16, 32, 64, 128)

# The checks below run on every call, single-token ones too: each looks at a
# tensor once, and takes its time only when something is wrong.

def _dtype(x, name):
    dt = x.dtype
    if dt is torch.bfloat16:
        return 0
    if dt is torch.float32:
        return 1
    raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {dt}")


def _is(name, t, shape, dtype, dev):
    """Refuses a tensor of another type, shape or device."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} is on {t.device}: all tensors must share one device")


def _dense(name, t, shape, dtype, dev):
    """Address of a contiguous tensor of this type and shape (None: None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.shape == shape:
        return t.data_ptr()
    _is(name, t, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor, got shape {tuple(t.shape)} strides {t.stride()}")
    return t.data_ptr()


def _aligned(*tensors):
    """Inputs that the kernels read 16 bytes at a time, those that start
    elsewhere as copies: a slice of a joined gradient, of a state cache or of a
    joined weight, with rows of any width, may.  (Held by the caller until its
    launch.)"""
    return [t.clone() if t is not None and t.data_ptr() & 15 and t.is_contiguous() else t for t in tensors]


_device = torch._C._cuda_getDevice


def _on_gpu(dev, x):
    """The library launches on the current device: a tensor of another one is refused."""
    if dev < 0:
        raise ValueError(f"expected a CUDA tensor, got one on {x.device}")
    if dev != _device():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{_device()}: "
                         "call under torch.cuda.device")


_current = torch._C._cuda_getCurrentRawStream


def _new(x):
    """A contiguous tensor of x's shape and type (the quickest call that gives one)."""
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _rows(x, width, inner=1):
    """(address, row stride) of an activation whose last `inner` dimensions
    form a dense row of `width` elements and whose rows are evenly spaced."""
    if x.is_contiguous():
        return x.data_ptr(), width
    shape, strides = x.shape, x.stride()
    if inner == 1 and len(shape) == 2 and strides[1] == 1 and strides[0] >= width:
        return x.data_ptr(), strides[0]
    dense = width
    for k in range(len(shape) - inner, len(shape)):
        dense //= max(shape[k], 1)
        if strides[k] != dense and shape[k] != 1:
            raise ValueError(f"expected dense rows, got shape {tuple(shape)} strides {strides}")
    row = step = None
    for k in range(len(shape) - inner - 1, -1, -1):
        if shape[k] == 1:
            continue
        if row is None:
            row = strides[k]
        elif strides[k] != step:
            raise ValueError(f"expected evenly spaced rows, got shape {tuple(shape)} strides {strides}")
        step = strides[k] * shape[k]
    if row is None:
        row = width
    if row < width:
        raise ValueError(f"expected rows apart from each other, got shape {tuple(shape)} strides {strides}")
    return x.data_ptr(), row


def _activation(name, allowed=("none", "silu")):
    if name not in _ACTIVATIONS or (name or "none") not in allowed:
        raise ValueError(f"activation must be one of {allowed}, got {name!r}")
    return _ACTIVATIONS[name]


def _sequences(x, cu_seqlens, dev, name):
    """(number of sequences, address of the offsets) of a (B, T, ...) activation."""
    if cu_seqlens is None:
        return x.shape[0], None
    if cu_seqlens.dtype is not torch.int32:
        raise ValueError(f"cu_seqlens must be int32, got {cu_seqlens.dtype}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 offsets")
    if x.shape[0] != 1:
        raise ValueError(f"packed inputs must have batch extent 1, got {name} of shape {tuple(x.shape)}")
    return cu_seqlens.numel() - 1, _dense("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, dev)


def _state(state, out_state, slots, batch, row, dtype, dev):
    """Addresses of a state cache, of where it goes, and of the slots; its rows."""
    if state.dim() != 3 or state.shape[1:] != row or (slots is None and state.shape[0] < batch):
        raise ValueError(f"state must be (S, {row[0]}, {row[1]}) with a row for each of the {batch}, "
                         f"got shape {tuple(state.shape)}")
    shape = state.shape
    to = state if out_state is None else out_state
    at = _dense("state", state, shape, dtype, dev)
    return (at, at if to is state else _dense("out_state", to, shape, dtype, dev),
            None if slots is None else _dense("slots", slots, (batch,), torch.int32, dev), shape[0])


# ----------------------------------------------------------------------------
# short causal convolution
# ----------------------------------------------------------------------------

def _taps(weight, D):
    if weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError(f"weight must be (D, W) with D = {D}, got shape {tuple(weight.shape)}")
    W = weight.shape[1]
    if not 2 <= W <= 4:
        raise ValueError(f"weight must have 2, 3 or 4 taps, got {W}")
    return W


def _conv_args(x, weight, bias, activation, initial_state, cu_seqlens):
    if x.dim() != 3:
        raise ValueError(f"x must be (B, T, D), got shape {tuple(x.shape)}")
    dtype, dev = _dtype(x, "x"), x.get_device()
    act = _activation(activation)
    T, D = x.shape[1:]
    W = _taps(weight, D)
    N, cu = _sequences(x, cu_seqlens, dev, "x")
    ptrs = (_dense("weight", weight, (D, W), torch.float32, dev), _dense("bias", bias, (D,), torch.float32, dev),
            _dense("initial_state", initial_state, (N, W - 1, D), x.dtype, dev), cu)
    _on_gpu(dev, x)
    return dev, (N, T, D, W, act, dtype), (*_rows(x, D), *ptrs)


def short_conv_fwd(x, weight, bias=None, activation="silu", initial_state=None, cu_seqlens=None,
                   output_final_state=False, stream=None):
    """Causal convolution of every channel over its last W tokens: x (B, T, D),
    weight (D, W), bias (D), initial_state (N, W - 1, D) in x's dtype (the
    inputs before each sequence).  Returns (y (B, T, D), final_state or None)."""
    if stream is not None:
        return _on_stream(short_conv_fwd, locals())
    weight, bias, initial_state = _aligned(weight, bias, initial_state)
    dev, dims, args = _conv_args(x, weight, bias, activation, initial_state, cu_seqlens)
    y = _new(x)
    fs = None
    if output_final_state:
        fs = x.new_empty((dims[0], dims[3] - 1, dims[2])) if initial_state is None else torch.empty_like(initial_state)
    _check(load().gdn_conv_fwd(*args, y.data_ptr(), None if fs is None else fs.data_ptr(), *dims, _current(dev)),
           "gdn_conv_fwd")
    return y, fs


def short_conv_bwd(x, weight, d_out, bias=None, activation="silu", initial_state=None, cu_seqlens=None,
                   d_final_state=None, stream=None):
    """Gradients of short_conv_fwd: a dict of dx, dweight, dbias (with a bias)
    and d_initial_state (with an initial state)."""
    if stream is not None:
        return _on_stream(short_conv_bwd, locals())
    weight, bias, initial_state, d_out, d_final_state = _aligned(weight, bias, initial_state, d_out, d_final_state)
    dev, dims, args = _conv_args(x, weight, bias, activation, initial_state, cu_seqlens)
    N, T, D, W = dims[:4]
    dout = _dense("d_out", d_out, x.shape, x.dtype, dev)
    dfs = _dense("d_final_state", d_final_state, (N, W - 1, D), x.dtype, dev)
    res = {"dx": _new(x), "dweight": torch.empty_like(weight)}
    if bias is not None:
        res["dbias"] = torch.empty_like(bias)
    if initial_state is not None:
        res["d_initial_state"] = torch.empty_like(initial_state)
    lib = load()
    nbytes = lib.gdn_conv_bwd_workspace_size(N, T, D, W, int(cu_seqlens is not None))
    ws = _workspace(nbytes, x.device)
    _check(lib.gdn_conv_bwd(*args, dout, dfs, res["dx"].data_ptr(), res["dweight"].data_ptr(), _out(res, "dbias"),
                            _out(res, "d_initial_state"), *dims, ws.data_ptr(), nbytes, _current(dev)),
           "gdn_conv_bwd")
    return res


def _out(res, name):
    t = res.get(name)
    return None if t is None else t.data_ptr()


def short_conv_step(x, state, weight, bias=None, activation="silu", slots=None, out_state=None, stream=None):
    """One token per row: x (B, D) and a state cache (S, W - 1, D), updated in
    place or into out_state.  slots (B, int32): the cache row of each batch row
    (negative: an idle row, whose output is zero); by default row b.  Returns y
    (B, D)."""
    if stream is not None:
        return _on_stream(short_conv_step, locals())
    if x.dim() != 2:
        raise ValueError(f"x must be (B, D), got shape {tuple(x.shape)}")
    weight, bias = _aligned(weight, bias)
    dtype, dev = _dtype(x, "x"), x.get_device()
    act = _activation(activation)
    B, D = x.shape
    W = _taps(weight, D)
    w = _dense("weight", weight, (D, W), torch.float32, dev)
    b = _dense("bias", bias, (D,), torch.float32, dev)
    at, to, sl, S = _state(state, out_state, slots, B, (W - 1, D), x.dtype, dev)
    _on_gpu(dev, x)
    y = _new(x)
    _check(load().gdn_conv_step(*_rows(x, D), w, b, at, to, sl, y.data_ptr(), B, S, D, W, act, dtype,
                             _current(dev)), "gdn_conv_step")
    return y


# ----------------------------------------------------------------------------
# selective state space scan
# ----------------------------------------------------------------------------

def _scan_args(u, dt, A, B, C, D, z, dt_bias, softplus):
    """Checks shared by the scan and its step (u of 3 or 2 dimensions)."""
    dtype, dev, kind = _dtype(u, "u"), u.get_device(), u.dtype
    shape = u.shape
    width = shape[-1]
    if A.dim() != 2 or A.shape[0] != width:
        raise ValueError(f"A must be (D, N) with D = {width}, got shape {tuple(A.shape)}")
    N = A.shape[1]
    if N not in STATE_SIZES:
        raise ValueError(f"the state size must be one of {STATE_SIZES}, got {N}")
    _is("dt", dt, shape, kind, dev)
    if z is not None:
        _is("z", z, shape, kind, dev)
    if B.dim() != len(shape) + 1:
        raise ValueError(f"B must be {tuple(shape[:-1])} + (G, N), got shape {tuple(B.shape)}")
    G = B.shape[-2]
    if G < 1 or width % G:
        raise ValueError(f"the {width} channels must divide into the {G} groups of B")
    rows = shape[:-1] + (G, N)
    _is("B", B, rows, kind, dev)
    _is("C", C, rows, kind, dev)
    a = _dense("A", A, (width, N), torch.float32, dev)
    d = _dense("D", D, (width,), torch.float32, dev)
    b = _dense("dt_bias", dt_bias, (width,), torch.float32, dev)
    pz, sz = (None, 0) if z is None else _rows(z, width)
    return (dev, (width, G, N, dtype),
            (*_rows(u, width), *_rows(dt, width), a, *_rows(B, G * N, 2), *_rows(C, G * N, 2), d, pz, sz, b,
             int(softplus)))


def ssm_scan_fwd(u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None,
                 cu_seqlens=None, output_final_state=True, save_for_backward=False, stream=None):
    """Selective state space scan: u, dt, z (B, T, D); A (D, N); B, C
    (B, T, G, N); D, dt_bias (D); initial_state (N_seq, D, N) fp32.  Returns
    (out, final_state or None), or (out, final_state, saved) with
    save_for_backward (the states ssm_scan_bwd starts from)."""
    if stream is not None:
        return _on_stream(ssm_scan_fwd, locals())
    if u.dim() != 3:
        raise ValueError(f"u must be (B, T, D), got shape {tuple(u.shape)}")
    A, D, dt_bias, initial_state = _aligned(A, D, dt_bias, initial_state)
    dev, dims, args = _scan_args(u, dt, A, B, C, D, z, dt_bias, dt_softplus)
    nseq, cu = _sequences(u, cu_seqlens, dev, "u")
    width, G, N, dtype = dims
    T, varlen = u.shape[1], int(cu_seqlens is not None)
    h0 = _dense("initial_state", initial_state, (nseq, width, N), torch.float32, dev)
    _on_gpu(dev, u)
    out = _new(u)
    fs = None
    if output_final_state:
        fs = A.new_empty((nseq, width, N)) if initial_state is None else torch.empty_like(initial_state)
    lib = load()
    saved, sbytes = None, 0
    if save_for_backward:
        sbytes = lib.gdn_ssm_saved_size(nseq, T, width, N, varlen)
        saved = torch.empty(sbytes, dtype=torch.uint8, device=u.device)
    nbytes = lib.gdn_ssm_fwd_workspace_size(nseq, T, width, G, N, varlen)
    ws = _workspace(nbytes, u.device)
    _check(lib.gdn_ssm_fwd(*args, h0, cu, out.data_ptr(), None if fs is None else fs.data_ptr(),
                           None if saved is None else saved.data_ptr(), sbytes, nseq, T, *dims,
                           None if ws is None else ws.data_ptr(), nbytes, _current(dev)), "gdn_ssm_fwd")
    return (out, fs, saved) if save_for_backward else (out, fs)


def ssm_scan_bwd(u, dt, A, B, C, d_out, saved, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None,
                 cu_seqlens=None, d_final_state=None, stream=None):
    """Gradients of ssm_scan_fwd from the same inputs and the `saved` that it
    returned: a dict of du, ddt, dA, dB, dC, and dD, dz, ddt_bias and
    d_initial_state for those that were given."""
    if stream is not None:
        return _on_stream(ssm_scan_bwd, locals())
    if u.dim() != 3:
        raise ValueError(f"u must be (B, T, D), got shape {tuple(u.shape)}")
    A, D, dt_bias, d_out, d_final_state = _aligned(A, D, dt_bias, d_out, d_final_state)
    dev, dims, args = _scan_args(u, dt, A, B, C, D, z, dt_bias, dt_softplus)
    nseq, cu = _sequences(u, cu_seqlens, dev, "u")
    width, G, N, dtype = dims
    T, varlen = u.shape[1], int(cu_seqlens is not None)
    dout = _dense("d_out", d_out, u.shape, u.dtype, dev)
    _dense("initial_state", initial_state, (nseq, width, N), torch.float32, dev)
    dfs = _dense("d_final_state", d_final_state, (nseq, width, N), torch.float32, dev)
    if saved.dtype is not torch.uint8 or saved.get_device() != dev or not saved.is_contiguous():
        raise ValueError("saved must be the uint8 buffer that the saving forward returned, on u's device")
    _on_gpu(dev, u)
    res = {"du": _new(u), "ddt": _new(u), "dA": torch.empty_like(A),
           "dB": _new(B), "dC": _new(C)}
    if D is not None:
        res["dD"] = torch.empty_like(D)
    if z is not None:
        res["dz"] = _new(u)
    if dt_bias is not None:
        res["ddt_bias"] = torch.empty_like(dt_bias)
    if initial_state is not None:
        res["d_initial_state"] = torch.empty_like(initial_state)
    lib = load()
    nbytes = lib.gdn_ssm_bwd_workspace_size(nseq, T, width, G, N, varlen)
    ws = _workspace(nbytes, u.device)
    out = [_out(res, k) for k in ("du", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "d_initial_state")]
    _check(lib.gdn_ssm_bwd(*args, cu, dout, dfs, saved.data_ptr(), saved.numel(), *out, nseq, T, *dims,
                           ws.data_ptr(), nbytes, _current(dev)), "gdn_ssm_bwd")
    return res


def ssm_scan_step(u, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=True, slots=None, out_state=None,
                  stream=None):
    """One token per row: u, dt, z (B, D), B, C (B, G, N) and a state cache
    (S, D, N) fp32, updated in place or into out_state; slots as in
    short_conv_step.  Returns out (B, D)."""
    if stream is not None:
        return _on_stream(ssm_scan_step, locals())
    if u.dim() != 2:
        raise ValueError(f"u must be (B, D), got shape {tuple(u.shape)}")
    A, D, dt_bias = _aligned(A, D, dt_bias)
    dev, dims, args = _scan_args(u, dt, A, B, C, D, z, dt_bias, dt_softplus)
    batch, width = u.shape
    at, to, sl, S = _state(state, out_state, slots, batch, (width, dims[2]), torch.float32, dev)
    _on_gpu(dev, u)
    out = _new(u)
    _check(load().gdn_ssm_step(*args, at, to, sl, out.data_ptr(), batch, S, *dims, _current(dev)), "gdn_ssm_step")
    return out


# ----------------------------------------------------------------------------
# group norm with an activation
# ----------------------------------------------------------------------------

def _norm_args(x, weight, bias, gate, groups, activation):
    act = _activation(activation, ("none", "silu", "sigmoid"))
    shape = x.shape
    if len(shape) < 2:
        raise ValueError(f"x must be (..., C) with at least one row dimension, got shape {tuple(shape)}")
    dtype, dev, C = _dtype(x, "x"), x.get_device(), shape[-1]
    if groups < 1 or C < 1 or C % groups:
        raise ValueError(f"the {C} channels must divide into the {groups} groups")
    w = _dense("weight", weight, (C,), torch.float32, dev)
    b = _dense("bias", bias, (C,), torch.float32, dev)
    pg, sg = None, 0
    if gate is not None:
        _is("gate", gate, shape, x.dtype, dev)
        pg, sg = _rows(gate, C)
    _on_gpu(dev, x)
    return dev, act, dtype, x.numel() // C, C, (*_rows(x, C), pg, sg, w, b)


def group_norm_fwd(x, weight=None, bias=None, gate=None, groups=1, eps=1e-6, activation="silu", center=False,
                   gate_first=False, stream=None):
    """Norm of every row's groups of channels, with a gate or an activation:
    x, gate (..., C), weight, bias (C).  The statistics are those of one row
    (token), not of all positions of a sample as in torch.nn.GroupNorm.  center=False is the RMS norm, True
    subtracts the mean.  With a gate: norm(x) act(gate), or norm(x act(gate))
    with gate_first; without one: act(norm(x)).  Returns y (..., C)."""
    if stream is not None:
        return _on_stream(group_norm_fwd, locals())
    weight, bias = _aligned(weight, bias)
    dev, act, dtype, rows, C, args = _norm_args(x, weight, bias, gate, groups, activation)
    y = _new(x)
    _check(load().gdn_norm_fwd(*args, y.data_ptr(), rows, C, groups, eps, act, int(center), int(gate_first), dtype,
                            _current(dev)), "gdn_norm_fwd")
    return y


def group_norm_bwd(x, d_out, weight=None, bias=None, gate=None, groups=1, eps=1e-6, activation="silu", center=False,
                   gate_first=False, stream=None):
    """Gradients of group_norm_fwd: a dict of dx, and dweight, dbias and dgate
    for those that were given."""
    if stream is not None:
        return _on_stream(group_norm_bwd, locals())
    weight, bias, d_out = _aligned(weight, bias, d_out)
    dev, act, dtype, rows, C, args = _norm_args(x, weight, bias, gate, groups, activation)
    dout = _dense("d_out", d_out, x.shape, x.dtype, dev)
    res = {"dx": _new(x)}
    if gate is not None:
        res["dgate"] = _new(x)
    if weight is not None:
        res["dweight"] = torch.empty_like(weight)
    if bias is not None:
        res["dbias"] = torch.empty_like(bias)
    lib = load()
    nbytes = 0
    if weight is not None or bias is not None:
        nbytes = lib.gdn_norm_bwd_workspace_size(rows, C, groups, dtype)
    ws = _workspace(nbytes, x.device)
    _check(lib.gdn_norm_bwd(*args, dout, res["dx"].data_ptr(), _out(res, "dgate"), _out(res, "dweight"),
                            _out(res, "dbias"), rows, C, groups, eps, act, int(center), int(gate_first), dtype,
                            None if ws is None else ws.data_ptr(), nbytes, _current(dev)), "gdn_norm_bwd")
    return res


# ----------------------------------------------------------------------------
# autograd
# ----------------------------------------------------------------------------

_FUNCTIONS = {}


def _functions():
    if _FUNCTIONS:
        return _FUNCTIONS

    def dense(g, like):
        return g.to(like.dtype).contiguous()

    class ShortConv(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, initial_state, activation, cu_seqlens):
            y, fs = short_conv_fwd(x, weight, bias, activation, initial_state, cu_seqlens, output_final_state=True)
            ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
            ctx.activation = activation
            ctx.set_materialize_grads(False)
            return y, fs

        @staticmethod
        @first_order
        def backward(ctx, saved_tensors, d_out, d_fs):
            x, weight, bias, initial_state, cu_seqlens = saved_tensors
            d_out = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if d_out is None else dense(d_out, x)
            r = short_conv_bwd(x, weight, d_out, bias, ctx.activation, initial_state, cu_seqlens,
                               None if d_fs is None else dense(d_fs, x))
            return r["dx"], r["dweight"], r.get("dbias"), r.get("d_initial_state"), None, None

    class SsmScan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, u, dt, A, B, C, D, z, dt_bias, initial_state, dt_softplus, cu_seqlens):
            out, fs, saved = ssm_scan_fwd(u, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens,
                                          save_for_backward=True)
            ctx.save_for_backward(u, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, saved)
            ctx.dt_softplus = dt_softplus
            ctx.set_materialize_grads(False)
            return out, fs

        @staticmethod
        @first_order
        def backward(ctx, saved_tensors, d_out, d_fs):
            u, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, saved = saved_tensors
            d_out = torch.zeros(u.shape, dtype=u.dtype, device=u.device) if d_out is None else dense(d_out, u)
            d_fs = None if d_fs is None else d_fs.to(torch.float32).contiguous()
            r = ssm_scan_bwd(u, dt, A, B, C, d_out, saved, D, z, dt_bias, ctx.dt_softplus, initial_state, cu_seqlens,
                             d_fs)
            return (r["du"], r["ddt"], r["dA"], r["dB"], r["dC"], r.get("dD"), r.get("dz"), r.get("ddt_bias"),
                    r.get("d_initial_state"), None, None)

    class GroupNorm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, weight, bias, gate, groups, eps, activation, center, gate_first):
            ctx.save_for_backward(x, weight, bias, gate)
            ctx.rest = (groups, eps, activation, center, gate_first)
            return group_norm_fwd(x, weight, bias, gate, *ctx.rest)

        @staticmethod
        @first_order
        def backward(ctx, saved_tensors, d_out):
            x, weight, bias, gate = saved_tensors
            r = group_norm_bwd(x, dense(d_out, x), weight, bias, gate, *ctx.rest)
            return (r["dx"], r.get("dweight"), r.get("dbias"), r.get("dgate")) + (None,) * 5

    _FUNCTIONS.update(conv=ShortConv, scan=SsmScan, norm=GroupNorm)
    return _FUNCTIONS


def short_conv(x, weight, bias=None, activation="silu", initial_state=None, cu_seqlens=None):
    """short_conv_fwd with autograd (x, weight, bias, initial_state).  Returns
    (y, final_state)."""
    return _functions()["conv"].apply(x, weight, bias, initial_state, activation, cu_seqlens)


def ssm_scan(u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None, cu_seqlens=None):
    """ssm_scan_fwd with autograd (every tensor but cu_seqlens).  Returns
    (out, final_state).  The states for the backward are kept where one can
    follow: some input needs a gradient and grad mode is on."""
    if not (torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in
                                            (u, dt, A, B, C, D, z, dt_bias, initial_state))):
        return ssm_scan_fwd(u, dt, A, B, C, D, z, dt_bias, dt_softplus, initial_state, cu_seqlens)
    return _functions()["scan"].apply(u, dt, A, B, C, D, z, dt_bias, initial_state, dt_softplus, cu_seqlens)


def group_norm(x, weight=None, bias=None, gate=None, groups=1, eps=1e-6, activation="silu", center=False,
               gate_first=False):
    """group_norm_fwd with autograd (x, weight, bias, gate)."""
    return _functions()["norm"].apply(x, weight, bias, gate, groups, eps, activation, center, gate_first)
