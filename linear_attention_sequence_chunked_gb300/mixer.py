"""The operators around the recurrence of a mixer layer: a short causal
convolution, the selective state space scan, and the group norm with an
activation; for prompts, for training, and token by token.

As in gdn.py, nothing is computed here: arguments are checked and handed to
the CUDA kernels of ``_build/libgdn.so`` (include/gdn.h has the formulas and
layouts), without a CPU fallback.  ``*_fwd`` / ``*_bwd`` / ``*_step`` allocate
their outputs and workspaces with torch; short_conv, ssm_scan and group_norm
are the same forwards and backwards behind torch.autograd.

Activations are channels last and bf16 or fp32, one type per call; parameters
and the states of the scan are fp32.  The activation inputs x, gate, u, dt, z,
B and C may be slices of a wider projection: any tensor whose rows are dense
and evenly spaced.  Other inputs are contiguous.
"""

from __future__ import annotations

from .gdn import _check, _ptr, _stream, _workspace, load

_ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "sigmoid": 2}
STATE_SIZES = (8, 16, 32, 64, 128)


def _torch():
    import torch
    return torch


def _dtype(x, name):
    torch = _torch()
    if x.dtype == torch.bfloat16:
        return 0
    if x.dtype == torch.float32:
        return 1
    raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {x.dtype}")


def _rows(x, inner=1):
    """(address, row stride) of an activation whose last `inner` dimensions
    form a dense row and whose rows are evenly spaced."""
    if x.device.type != "cuda":
        raise ValueError(f"expected a CUDA tensor, got one on {x.device}")
    width = 1
    if not x.is_contiguous():
        shape, strides = x.shape, x.stride()
        lead = x.dim() - inner
        for k in range(x.dim() - 1, lead - 1, -1):
            if shape[k] != 1 and strides[k] != width:
                raise ValueError(f"expected dense rows, got shape {tuple(shape)} strides {strides}")
            width *= shape[k]
        row = step = None
        for k in range(lead - 1, -1, -1):
            if shape[k] == 1:
                continue
            if row is None:
                row = step = strides[k]
            elif strides[k] != step:
                raise ValueError(f"expected evenly spaced rows, got shape {tuple(shape)} strides {strides}")
            step = strides[k] * shape[k]
        if row is None:
            row = width
        if row < width and x.numel():
            raise ValueError(f"expected rows apart from each other, got shape {tuple(shape)} strides {strides}")
        return x.data_ptr(), max(row, width)
    for k in range(1, inner + 1):
        width *= x.shape[-k]
    return x.data_ptr(), width


def _same(name, t, shape, dtype, device):
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}: all tensors must share one device ({device})")


def _activation(name, allowed=("none", "silu")):
    if name not in _ACTIVATIONS or (name or "none") not in allowed:
        raise ValueError(f"activation must be one of {allowed}, got {name!r}")
    return _ACTIVATIONS[name]


def _sequences(x, cu_seqlens, name):
    """(N, B of the C ABI) of a (B, T, ...) activation."""
    if cu_seqlens is None:
        return x.shape[0]
    torch = _torch()
    if cu_seqlens.dtype != torch.int32:
        raise ValueError(f"cu_seqlens must be int32, got {cu_seqlens.dtype}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 offsets")
    if cu_seqlens.device != x.device:
        raise ValueError(f"cu_seqlens is on {cu_seqlens.device}: all tensors must share one device ({x.device})")
    if x.shape[0] != 1:
        raise ValueError(f"packed inputs must have batch extent 1, got {name} of shape {tuple(x.shape)}")
    return cu_seqlens.numel() - 1


def _check_slots(slots, batch, device):
    if slots is not None:
        _same("slots", slots, (batch,), _torch().int32, device)


# ----------------------------------------------------------------------------
# short causal convolution
# ----------------------------------------------------------------------------

def _conv_args(x, weight, bias, initial_state, cu_seqlens):
    torch = _torch()
    if x.dim() != 3:
        raise ValueError(f"x must be (B, T, D), got shape {tuple(x.shape)}")
    dtype = _dtype(x, "x")
    B, T, D = x.shape
    if weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError(f"weight must be (D, W) with D = {D}, got shape {tuple(weight.shape)}")
    W = weight.shape[1]
    if W not in (2, 3, 4):
        raise ValueError(f"weight must have 2, 3 or 4 taps, got {W}")
    N = _sequences(x, cu_seqlens, "x")
    _same("weight", weight, (D, W), torch.float32, x.device)
    _same("bias", bias, (D,), torch.float32, x.device)
    _same("initial_state", initial_state, (N, W - 1, D), x.dtype, x.device)
    return dtype, N, T, D, W


def short_conv_fwd(x, weight, bias=None, activation="silu", initial_state=None, cu_seqlens=None,
                   output_final_state=False, stream=None):
    """Causal convolution of every channel over its last W tokens: x (B, T, D),
    weight (D, W), bias (D), initial_state (N, W - 1, D) in x's dtype (the
    inputs before each sequence).  Returns (y (B, T, D), final_state or None)."""
    torch = _torch()
    dtype, N, T, D, W = _conv_args(x, weight, bias, initial_state, cu_seqlens)
    act = _activation(activation)
    px, sx = _rows(x)
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    fs = torch.empty((N, W - 1, D), dtype=x.dtype, device=x.device) if output_final_state else None
    _check(load().gdn_conv_fwd(px, sx, _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens), _ptr(y),
                               _ptr(fs), N, T, D, W, act, dtype, _stream(stream)), "gdn_conv_fwd")
    return y, fs


def short_conv_bwd(x, weight, d_out, bias=None, activation="silu", initial_state=None, cu_seqlens=None,
                   d_final_state=None, stream=None):
    """Gradients of short_conv_fwd: a dict of dx, dweight, dbias (with a bias)
    and d_initial_state (with an initial state)."""
    torch = _torch()
    dtype, N, T, D, W = _conv_args(x, weight, bias, initial_state, cu_seqlens)
    act = _activation(activation)
    _same("d_out", d_out, x.shape, x.dtype, x.device)
    _same("d_final_state", d_final_state, (N, W - 1, D), x.dtype, x.device)
    px, sx = _rows(x)
    dev = x.device
    res = {"dx": torch.empty(x.shape, dtype=x.dtype, device=dev),
           "dweight": torch.empty((D, W), dtype=torch.float32, device=dev)}
    if bias is not None:
        res["dbias"] = torch.empty((D,), dtype=torch.float32, device=dev)
    if initial_state is not None:
        res["d_initial_state"] = torch.empty((N, W - 1, D), dtype=x.dtype, device=dev)
    lib = load()
    nbytes = lib.gdn_conv_bwd_workspace_size(N, T, D, W, int(cu_seqlens is not None))
    ws = _workspace(nbytes, dev)
    _check(lib.gdn_conv_bwd(px, sx, _ptr(weight), _ptr(bias), _ptr(initial_state), _ptr(cu_seqlens), _ptr(d_out),
                            _ptr(d_final_state), _ptr(res["dx"]), _ptr(res["dweight"]), _ptr(res.get("dbias")),
                            _ptr(res.get("d_initial_state")), N, T, D, W, act, dtype, _ptr(ws), nbytes,
                            _stream(stream)), "gdn_conv_bwd")
    return res


def short_conv_step(x, state, weight, bias=None, activation="silu", slots=None, out_state=None, stream=None):
    """One token per row: x (B, D) and a state cache (S, W - 1, D), updated in
    place or into out_state.  slots (B, int32): the cache row of each batch row
    (negative: an idle row, whose output is zero); by default row b.  Returns y
    (B, D)."""
    torch = _torch()
    if x.dim() != 2:
        raise ValueError(f"x must be (B, D), got shape {tuple(x.shape)}")
    dtype = _dtype(x, "x")
    B, D = x.shape
    if weight.dim() != 2 or weight.shape[0] != D or weight.shape[1] not in (2, 3, 4):
        raise ValueError(f"weight must be (D, W) with D = {D} and 2, 3 or 4 taps, got shape {tuple(weight.shape)}")
    W = weight.shape[1]
    dev = x.device
    _same("weight", weight, (D, W), torch.float32, dev)
    _same("bias", bias, (D,), torch.float32, dev)
    _check_state(state, out_state, slots, B, (W - 1, D), x.dtype, dev)
    act = _activation(activation)
    px, sx = _rows(x)
    y = torch.empty((B, D), dtype=x.dtype, device=dev)
    _check(load().gdn_conv_step(px, sx, _ptr(weight), _ptr(bias), _ptr(state),
                                _ptr(state if out_state is None else out_state), _ptr(slots), _ptr(y), B,
                                state.shape[0], D, W, act, dtype, _stream(stream)), "gdn_conv_step")
    return y


def _check_state(state, out_state, slots, batch, row, dtype, device):
    if state.dim() != 3 or state.shape[1:] != row or (slots is None and state.shape[0] < batch):
        raise ValueError(f"state must be (S, {row[0]}, {row[1]}) with a row for each of the {batch}, "
                         f"got shape {tuple(state.shape)}")
    _same("state", state, state.shape, dtype, device)
    _same("out_state", out_state, state.shape, dtype, device)
    _check_slots(slots, batch, device)


# ----------------------------------------------------------------------------
# selective state space scan
# ----------------------------------------------------------------------------

def _scan_args(u, dt, A, B, C, D, z, dt_bias):
    """Checks shared by the scan and its step (u of 3 or 2 dimensions)."""
    torch = _torch()
    dtype = _dtype(u, "u")
    lead, width = u.shape[:-1], u.shape[-1]
    dev = u.device
    _same("dt", dt, u.shape, u.dtype, dev)
    _same("z", z, u.shape, u.dtype, dev)
    if A.dim() != 2 or A.shape[0] != width:
        raise ValueError(f"A must be (D, N) with D = {width}, got shape {tuple(A.shape)}")
    N = A.shape[1]
    if N not in STATE_SIZES:
        raise ValueError(f"the state size must be one of {STATE_SIZES}, got {N}")
    _same("A", A, (width, N), torch.float32, dev)
    if B.dim() != u.dim() + 1:
        raise ValueError(f"B must be {tuple(lead)} + (G, N), got shape {tuple(B.shape)}")
    G = B.shape[-2]
    if G < 1 or width % G:
        raise ValueError(f"the {width} channels must divide into the {G} groups of B")
    _same("B", B, lead + (G, N), u.dtype, dev)
    _same("C", C, lead + (G, N), u.dtype, dev)
    _same("D", D, (width,), torch.float32, dev)
    _same("dt_bias", dt_bias, (width,), torch.float32, dev)
    pz, sz = (None, 0) if z is None else _rows(z)
    return (dtype, width, G, N,
            (*_rows(u), *_rows(dt), _ptr(A), *_rows(B, 2), *_rows(C, 2), _ptr(D), pz, sz, _ptr(dt_bias)))


def ssm_scan_fwd(u, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None,
                 cu_seqlens=None, output_final_state=True, save_for_backward=False, stream=None):
    """Selective state space scan: u, dt, z (B, T, D); A (D, N); B, C
    (B, T, G, N); D, dt_bias (D); initial_state (N_seq, D, N) fp32.  Returns
    (out, final_state or None), or (out, final_state, saved) with
    save_for_backward (the states ssm_scan_bwd starts from)."""
    torch = _torch()
    if u.dim() != 3:
        raise ValueError(f"u must be (B, T, D), got shape {tuple(u.shape)}")
    nseq = _sequences(u, cu_seqlens, "u")
    dtype, width, G, N, args = _scan_args(u, dt, A, B, C, D, z, dt_bias)
    dev, T = u.device, u.shape[1]
    _same("initial_state", initial_state, (nseq, width, N), torch.float32, dev)
    varlen = int(cu_seqlens is not None)
    out = torch.empty(u.shape, dtype=u.dtype, device=dev)
    fs = torch.empty((nseq, width, N), dtype=torch.float32, device=dev) if output_final_state else None
    lib = load()
    saved, sbytes = None, 0
    if save_for_backward:
        sbytes = lib.gdn_ssm_saved_size(nseq, T, width, N, varlen)
        saved = torch.empty(sbytes, dtype=torch.uint8, device=dev)
    nbytes = lib.gdn_ssm_fwd_workspace_size(nseq, T, width, G, N, varlen)
    ws = _workspace(nbytes, dev)
    _check(lib.gdn_ssm_fwd(*args, int(dt_softplus), _ptr(initial_state), _ptr(cu_seqlens), _ptr(out), _ptr(fs),
                           _ptr(saved), sbytes, nseq, T, width, G, N, dtype, _ptr(ws), nbytes, _stream(stream)),
           "gdn_ssm_fwd")
    return (out, fs, saved) if save_for_backward else (out, fs)


def ssm_scan_bwd(u, dt, A, B, C, d_out, saved, D=None, z=None, dt_bias=None, dt_softplus=True, initial_state=None,
                 cu_seqlens=None, d_final_state=None, stream=None):
    """Gradients of ssm_scan_fwd from the same inputs and the `saved` that it
    returned: a dict of du, ddt, dA, dB, dC, and dD, dz, ddt_bias and
    d_initial_state for those that were given."""
    torch = _torch()
    if u.dim() != 3:
        raise ValueError(f"u must be (B, T, D), got shape {tuple(u.shape)}")
    nseq = _sequences(u, cu_seqlens, "u")
    dtype, width, G, N, args = _scan_args(u, dt, A, B, C, D, z, dt_bias)
    dev, T = u.device, u.shape[1]
    _same("d_out", d_out, u.shape, u.dtype, dev)
    _same("initial_state", initial_state, (nseq, width, N), torch.float32, dev)
    _same("d_final_state", d_final_state, (nseq, width, N), torch.float32, dev)
    if saved.dtype != torch.uint8 or saved.device != dev:
        raise ValueError("saved must be the uint8 buffer that the saving forward returned, on u's device")
    varlen = int(cu_seqlens is not None)
    f32 = {"dtype": torch.float32, "device": dev}
    res = {"du": torch.empty(u.shape, dtype=u.dtype, device=dev), "ddt": torch.empty(u.shape, dtype=u.dtype, device=dev),
           "dA": torch.empty((width, N), **f32), "dB": torch.empty(B.shape, dtype=u.dtype, device=dev),
           "dC": torch.empty(B.shape, dtype=u.dtype, device=dev)}
    if D is not None:
        res["dD"] = torch.empty((width,), **f32)
    if z is not None:
        res["dz"] = torch.empty(u.shape, dtype=u.dtype, device=dev)
    if dt_bias is not None:
        res["ddt_bias"] = torch.empty((width,), **f32)
    if initial_state is not None:
        res["d_initial_state"] = torch.empty((nseq, width, N), **f32)
    lib = load()
    nbytes = lib.gdn_ssm_bwd_workspace_size(nseq, T, width, G, N, varlen)
    ws = _workspace(nbytes, dev)
    out = [_ptr(res.get(k)) for k in ("du", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "d_initial_state")]
    _check(lib.gdn_ssm_bwd(*args, int(dt_softplus), _ptr(cu_seqlens), _ptr(d_out), _ptr(d_final_state), _ptr(saved),
                           saved.numel(), *out, nseq, T, width, G, N, dtype, _ptr(ws), nbytes, _stream(stream)),
           "gdn_ssm_bwd")
    return res


def ssm_scan_step(u, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus=True, slots=None, out_state=None,
                  stream=None):
    """One token per row: u, dt, z (B, D), B, C (B, G, N) and a state cache
    (S, D, N) fp32, updated in place or into out_state; slots as in
    short_conv_step.  Returns out (B, D)."""
    torch = _torch()
    if u.dim() != 2:
        raise ValueError(f"u must be (B, D), got shape {tuple(u.shape)}")
    dtype, width, G, N, args = _scan_args(u, dt, A, B, C, D, z, dt_bias)
    batch = u.shape[0]
    _check_state(state, out_state, slots, batch, (width, N), torch.float32, u.device)
    out = torch.empty((batch, width), dtype=u.dtype, device=u.device)
    _check(load().gdn_ssm_step(*args, int(dt_softplus), _ptr(state), _ptr(state if out_state is None else out_state),
                               _ptr(slots), _ptr(out), batch, state.shape[0], width, G, N, dtype, _stream(stream)),
           "gdn_ssm_step")
    return out


# ----------------------------------------------------------------------------
# group norm with an activation
# ----------------------------------------------------------------------------

def _norm_args(x, weight, bias, gate, groups):
    torch = _torch()
    if x.dim() < 2:
        raise ValueError(f"x must be (..., C) with at least one row dimension, got shape {tuple(x.shape)}")
    dtype = _dtype(x, "x")
    C = x.shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"the {C} channels must divide into the {groups} groups")
    _same("weight", weight, (C,), torch.float32, x.device)
    _same("bias", bias, (C,), torch.float32, x.device)
    _same("gate", gate, x.shape, x.dtype, x.device)
    pg, sg = (None, 0) if gate is None else _rows(gate)
    return dtype, x.numel() // C if C else 0, C, (*_rows(x), pg, sg, _ptr(weight), _ptr(bias))


def group_norm_fwd(x, weight=None, bias=None, gate=None, groups=1, eps=1e-6, activation="silu", center=False,
                   gate_first=False, stream=None):
    """Norm of every row's groups of channels, with a gate or an activation:
    x, gate (..., C), weight, bias (C).  center=False is the RMS norm, True
    subtracts the mean.  With a gate: norm(x) act(gate), or norm(x act(gate))
    with gate_first; without one: act(norm(x)).  Returns y (..., C)."""
    act = _activation(activation, ("none", "silu", "sigmoid"))
    dtype, rows, C, args = _norm_args(x, weight, bias, gate, groups)
    y = _torch().empty(x.shape, dtype=x.dtype, device=x.device)
    _check(load().gdn_norm_fwd(*args, _ptr(y), rows, C, groups, float(eps), act, int(center), int(gate_first), dtype,
                               _stream(stream)), "gdn_norm_fwd")
    return y


def group_norm_bwd(x, d_out, weight=None, bias=None, gate=None, groups=1, eps=1e-6, activation="silu", center=False,
                   gate_first=False, stream=None):
    """Gradients of group_norm_fwd: a dict of dx, and dweight, dbias and dgate
    for those that were given."""
    torch = _torch()
    act = _activation(activation, ("none", "silu", "sigmoid"))
    dtype, rows, C, args = _norm_args(x, weight, bias, gate, groups)
    _same("d_out", d_out, x.shape, x.dtype, x.device)
    dev = x.device
    res = {"dx": torch.empty(x.shape, dtype=x.dtype, device=dev)}
    if gate is not None:
        res["dgate"] = torch.empty(x.shape, dtype=x.dtype, device=dev)
    if weight is not None:
        res["dweight"] = torch.empty((C,), dtype=torch.float32, device=dev)
    if bias is not None:
        res["dbias"] = torch.empty((C,), dtype=torch.float32, device=dev)
    lib = load()
    nbytes = 0
    if weight is not None or bias is not None:
        nbytes = lib.gdn_norm_bwd_workspace_size(rows, C, groups, dtype)
    ws = _workspace(nbytes, dev)
    _check(lib.gdn_norm_bwd(*args, _ptr(d_out), _ptr(res["dx"]), _ptr(res.get("dgate")), _ptr(res.get("dweight")),
                            _ptr(res.get("dbias")), rows, C, groups, float(eps), act, int(center), int(gate_first),
                            dtype, _ptr(ws), nbytes, _stream(stream)), "gdn_norm_bwd")
    return res


# ----------------------------------------------------------------------------
# autograd
# ----------------------------------------------------------------------------

_FUNCTIONS = {}


def _functions():
    if _FUNCTIONS:
        return _FUNCTIONS
    torch = _torch()

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
        def backward(ctx, d_out, d_fs):
            x, weight, bias, initial_state, cu_seqlens = ctx.saved_tensors
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
        def backward(ctx, d_out, d_fs):
            u, dt, A, B, C, D, z, dt_bias, initial_state, cu_seqlens, saved = ctx.saved_tensors
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
        def backward(ctx, d_out):
            x, weight, bias, gate = ctx.saved_tensors
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
    (out, final_state)."""
    return _functions()["scan"].apply(u, dt, A, B, C, D, z, dt_bias, initial_state, dt_softplus, cu_seqlens)


def group_norm(x, weight=None, bias=None, gate=None, groups=1, eps=1e-6, activation="silu", center=False,
               gate_first=False):
    """group_norm_fwd with autograd (x, weight, bias, gate)."""
    return _functions()["norm"].apply(x, weight, bias, gate, groups, eps, activation, center, gate_first)
