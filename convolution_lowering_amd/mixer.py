"""Sequence-mixing operators: the short causal convolution, the gated delta
rule and the branch norm, over the C ABI of ``include/convlower_mixer.h``.

    conv1d_causal_fwd / _bwd / _step      silu(causal depthwise convolution)
    delta_rule_fwd / _bwd / _step         S <- e^g S + k (beta (v - e^g S'k))',  o = S'q
    branch_norm_fwd / _bwd                r = x + alpha act(gate) norm(y),  h = norm(r)
    conv1d_causal, delta_rule, branch_norm   the same, differentiable (once) by autograd

As in the package's convolution binding, Python only checks and marshals:
outputs and workspaces are allocated with torch on the stream the library
launches on (`stream`, else the current one of the tensors' device), and a
failing call raises ConvLowerError, ValueError or TypeError before anything is
launched.

Tokens of several sequences are packed along one axis: ``[T, ...]`` with
``cu_seqlens`` (int32, N + 1 offsets on the device), or ``[B, L, ...]`` for B
sequences of one length.  Tokens may be strided (slices of a wider packed
tensor); everything inside a token is dense.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from . import _check, lib

ACTS = {"none": 0, "silu": 1, "sigmoid": 2}
MAX_CONV_WIDTH, MAX_DK, MAX_DV, MAX_NORM_WIDTH = 8, 128, 256, 32768
# Every symbol include/convlower_mixer.h declares.
EXPORTS = ("conv1d_causal_fwd", "conv1d_causal_bwd_workspace_size", "conv1d_causal_bwd", "conv1d_causal_step",
           "delta_rule_fwd_workspace_size", "delta_rule_saved_size", "delta_rule_fwd",
           "delta_rule_bwd_workspace_size", "delta_rule_bwd", "delta_rule_step",
           "branch_norm_fwd", "branch_norm_bwd_workspace_size", "branch_norm_bwd")
_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_lib = None


def _mixer_lib():
    global _lib
    if _lib is None:
        L = lib()
        i, z, f, vp, l = ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_void_p, ctypes.c_int64
        size = ctypes.POINTER(z)
        L.conv1d_causal_fwd.argtypes = [vp, l] + [vp] * 6 + [l] + [i] * 5 + [vp]
        L.conv1d_causal_bwd_workspace_size.argtypes = [l, i, i, i, size]
        L.conv1d_causal_bwd.argtypes = [vp, l, vp, vp, l] + [vp] * 8 + [l] + [i] * 5 + [vp, vp, z]
        L.conv1d_causal_step.argtypes = [vp, l] + [vp] * 5 + [i] * 6 + [vp]
        for name in ("fwd_workspace_size", "saved_size", "bwd_workspace_size"):
            getattr(L, "delta_rule_" + name).argtypes = [l] + [i] * 6 + [size]
        L.delta_rule_fwd.argtypes = [vp, l] * 3 + [vp] * 6 + [l] + [i] * 5 + [f] + [i] * 3 + [vp, vp, z, vp, z]
        L.delta_rule_bwd.argtypes = ([vp, l, vp] + [vp, l] * 3 + [vp] * 4 + [z] + [vp] * 6 + [l] + [i] * 5 + [f] +
                                     [i] * 3 + [vp, vp, z])
        L.delta_rule_step.argtypes = [vp, l] * 3 + [vp] * 5 + [i] * 7 + [f] + [i] * 3 + [vp]
        L.branch_norm_fwd.argtypes = [vp] * 8 + [l, i, l, f, f, i, i, vp]
        L.branch_norm_bwd_workspace_size.argtypes = [l, i, l, size]
        L.branch_norm_bwd.argtypes = [vp] * 13 + [l, i, l, f, f, i, i, vp, vp, z]
        for name in EXPORTS:
            getattr(L, name).restype = i
        _lib = L
    return _lib


def _code(t, name):
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError(f"{name} has dtype {t.dtype}: float32, bfloat16 or float16 wanted")
    return c


def _dense(t, name, shape, dtype, device):
    """A contiguous device tensor of one shape; returns its address."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected {device}, a GPU")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _tokens(t, name, dims, dtype, device):
    """Address and token stride of a tensor whose last `dims` axes are one
    dense token, with one (packed) or two ([B, L]) token axes before them."""
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected {device}, a GPU")
    shape, stride = t.shape, t.stride()
    one, lead = 1, len(shape) - dims
    for a in range(len(shape) - 1, lead - 1, -1):
        if stride[a] != one and shape[a] != 1:
            raise ValueError(f"{name}: the axes of one token must be dense, strides are {tuple(stride)}")
        one *= shape[a]
    step = stride[lead - 1] if shape[lead - 1] > 1 else one
    if lead == 2 and shape[0] > 1:
        step = stride[0] if shape[1] == 1 else step
        if shape[1] > 1 and stride[0] != shape[1] * step:
            raise ValueError(f"{name}: its tokens do not lie at one stride, strides are {tuple(stride)}")
    if step < one and t.numel():
        raise ValueError(f"{name}: tokens overlap, strides are {tuple(stride)}")
    return t.data_ptr(), max(step, one)


def _packing(lead, cu_seqlens, device):
    """(tokens, sequences, address of the offsets) of the token axes `lead`."""
    if len(lead) == 2:
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens goes with packed tokens ([T, ...]), not with [B, L, ...]")
        if lead[0] < 1:
            raise ValueError("no sequences")
        return lead[0] * lead[1], lead[0], None
    if cu_seqlens is None:
        return lead[0], 1, None
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens: at least two int32 offsets wanted")
    return lead[0], cu_seqlens.numel() - 1, _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, device)


_HERE = contextlib.nullcontext()


def _on(stream, device):
    """Where outputs and workspaces are allocated and the launch is made: on
    the caller's stream, or the tensors' device and its current stream.  Where
    that device is torch's current one there is nothing to enter (and entering
    its stream again would cost a one-token call a third of its time)."""
    if stream is not None:
        return torch.cuda.stream(stream)
    return _HERE if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)


def _raw(stream, device):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def _act(act, allowed=("none", "silu")):
    if act not in allowed:
        raise ValueError(f"act {act!r}: one of {allowed} wanted")
    return ACTS[act]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _size(fn, *args):
    out = ctypes.c_size_t()
    _check(fn, getattr(_mixer_lib(), fn)(*args, ctypes.byref(out)))
    return out.value


def _bytes(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


# ------------------------------------------------------------ causal convolution


def _conv_args(x, w, bias, cu_seqlens, state, act):
    if x.dim() not in (2, 3) or w.dim() != 2:
        raise ValueError("x is [T, D] or [B, L, D], w [D, W]")
    D, W = w.shape
    if x.shape[-1] != D:
        raise ValueError(f"x has {x.shape[-1]} channels, w {D}")
    dt, dev = x.dtype, x.device
    code = _code(x, "x")
    xp, xs = _tokens(x, "x", 1, dt, dev)
    T, N, cu = _packing(x.shape[:-1], cu_seqlens, dev)
    return (code, xp, xs, _dense(w, "w", w.shape, dt, dev), _dense(bias, "bias", (D,), dt, dev),
            _dense(state, "state", (N, W - 1, D), dt, dev), cu, T, N, D, W, _act(act))


def conv1d_causal_fwd(x, w, bias=None, *, cu_seqlens=None, state=None, act="silu", want_state=False, stream=None):
    """y = act(bias + causal depthwise convolution of x with w) within each
    sequence; returns (y, state_out).

    x: [T, D] with cu_seqlens, or [B, L, D]; w: [D, W], w[:, -1] meets the
    token itself; bias: [D].  state: [N, W-1, D], the inputs before each
    sequence (zeros when None); state_out (want_state) the inputs that a later
    call on the same sequences takes as its state, else None."""
    code, xp, xs, wp, bp, sp, cu, T, N, D, W, a = _conv_args(x, w, bias, cu_seqlens, state, act)
    with _on(stream, x.device):
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        out = torch.empty((N, W - 1, D), dtype=x.dtype, device=x.device) if want_state else None
        _check("conv1d_causal_fwd",
               _mixer_lib().conv1d_causal_fwd(xp, xs, wp, bp, sp, cu, y.data_ptr(), _ptr(out), T, N, D, W, a, code,
                                              _raw(stream, x.device)))
    return y, out


def conv1d_causal_bwd(dy, x, w, bias=None, *, cu_seqlens=None, state=None, act="silu", dstate_out=None,
                      want_dstate=False, stream=None):
    """Gradients of conv1d_causal_fwd: (dx, dw, dbias, dstate); dbias is None
    without a bias, dstate None unless wanted.  dstate_out: the gradient of
    state_out, where it was used."""
    code, xp, xs, wp, bp, sp, cu, T, N, D, W, a = _conv_args(x, w, bias, cu_seqlens, state, act)
    if dy.shape != x.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, x {tuple(x.shape)}")
    dt, dev = x.dtype, x.device
    dyp, dys = _tokens(dy, "dy", 1, dt, dev)
    dso = _dense(dstate_out, "dstate_out", (N, W - 1, D), dt, dev)
    with _on(stream, dev):
        dx = torch.empty(x.shape, dtype=dt, device=dev)
        dw = torch.empty((D, W), dtype=dt, device=dev)
        db = torch.empty(D, dtype=dt, device=dev) if bias is not None else None
        ds = torch.empty((N, W - 1, D), dtype=dt, device=dev) if want_dstate else None
        ws = _bytes(_size("conv1d_causal_bwd_workspace_size", T, N, D, W), dev)
        _check("conv1d_causal_bwd",
               _mixer_lib().conv1d_causal_bwd(dyp, dys, dso, xp, xs, wp, bp, sp, cu, dx.data_ptr(), dw.data_ptr(),
                                              _ptr(db), _ptr(ds), T, N, D, W, a, code, _raw(stream, dev), _ptr(ws),
                                              ws.numel() if ws is not None else 0))
    return dx, dw, db, ds


def conv1d_causal_step(x, w, bias, pool, slots=None, *, act="silu", out=None, stream=None):
    """One token for each request: y [R, D] from x [R, D] and the requests'
    last inputs pool[slots] ([P, W-1, D], moved on in place).  slots: int32
    [R], all different; a slot outside the pool is padding (y zero).  None:
    request r is slot r."""
    D, W = w.shape
    R, dt, dev = x.shape[0], x.dtype, x.device
    code = _code(x, "x")
    if x.dim() != 2 or x.shape[1] != D or pool.dim() != 3:
        raise ValueError("x is [R, D], pool [P, W-1, D]")
    xp, xs = _tokens(x, "x", 1, dt, dev)
    P = pool.shape[0]
    args = (xp, xs, _dense(w, "w", w.shape, dt, dev), _dense(bias, "bias", (D,), dt, dev),
            _dense(pool, "pool", (P, W - 1, D), dt, dev), _dense(slots, "slots", (R,), torch.int32, dev))
    with _on(stream, dev):
        y = torch.empty((R, D), dtype=dt, device=dev) if out is None else out
        _check("conv1d_causal_step",
               _mixer_lib().conv1d_causal_step(*args, _dense(y, "out", (R, D), dt, dev), R, P, D, W, _act(act), code,
                                               _raw(stream, dev)))
    return y


# -------------------------------------------------------------- gated delta rule


def _delta_args(q, k, v, g, beta):
    """Addresses, strides and sizes of one call's inputs."""
    d = v.dim()
    if d not in (3, 4) or q.dim() != d or k.shape != q.shape or q.shape[:-2] != v.shape[:-2]:
        raise ValueError("q, k are [T, Hk, dk] (or [B, L, Hk, dk]), v [T, Hv, dv]")
    Hk, dk = q.shape[-2:]
    Hv, dv = v.shape[-2:]
    if Hk < 1 or Hv % Hk:
        raise ValueError(f"{Hv} value heads are no multiple of {Hk} query/key heads")
    dt, dev = q.dtype, q.device
    code = _code(q, "q")
    if beta.dtype != dt and beta.dtype != torch.float32:
        raise TypeError(f"beta has dtype {beta.dtype}, expected {dt} or float32")
    heads = v.shape[:-1]
    return ((*_tokens(q, "q", 2, dt, dev), *_tokens(k, "k", 2, dt, dev), *_tokens(v, "v", 2, dt, dev),
             _dense(g, "g", heads, torch.float32, dev), _dense(beta, "beta", heads, beta.dtype, dev)),
            (Hk, Hv, dk, dv), code, _CODES[beta.dtype])


def delta_rule_fwd(q, k, v, g, beta, *, cu_seqlens=None, state=None, scale=None, qk_norm=False, want_state=False,
                   save=False, stream=None):
    """The gated delta rule along each sequence; returns (o, state_out, saved).

        S <- exp(g) S;  u = beta (v - S'k);  S <- S + k u';  o = scale S'q

    q, k: [T, Hk, dk] with cu_seqlens, or [B, L, Hk, dk]; v: [T, Hv, dv], Hv a
    multiple of Hk (value head h reads q/k head h // (Hv // Hk)); g: fp32
    [T, Hv], log decays; beta: [T, Hv].  state: fp32 [N, Hv, dk, dv] (zeros
    when None); state_out (want_state) the state after each sequence.  scale:
    dk ** -0.5 when None.  qk_norm: q and k are divided by their 2-norms.
    save: what delta_rule_bwd of the same call takes as `saved`."""
    ptrs, sizes, code, bcode = _delta_args(q, k, v, g, beta)
    Hk, Hv, dk, dv = sizes
    dev = q.device
    T, N, cu = _packing(v.shape[:-2], cu_seqlens, dev)
    sp = _dense(state, "state", (N, Hv, dk, dv), torch.float32, dev)
    scale = dk ** -0.5 if scale is None else scale
    with _on(stream, dev):
        o = torch.empty(v.shape, dtype=q.dtype, device=dev)
        out = torch.empty((N, Hv, dk, dv), dtype=torch.float32, device=dev) if want_state else None
        ws = _bytes(_size("delta_rule_fwd_workspace_size", T, N, *sizes, code), dev)
        saved = _bytes(max(16, _size("delta_rule_saved_size", T, N, *sizes, code)), dev) if save else None
        _check("delta_rule_fwd",
               _mixer_lib().delta_rule_fwd(*ptrs, sp, cu, o.data_ptr(), _ptr(out), T, N, *sizes, scale, qk_norm, code,
                                           bcode, _raw(stream, dev), _ptr(ws), ws.numel() if ws is not None else 0,
                                           _ptr(saved), saved.numel() if save else 0))
    return o, out, saved


def delta_rule_bwd(do, q, k, v, g, beta, saved, *, cu_seqlens=None, scale=None, qk_norm=False, dstate_out=None,
                   want_dstate=False, stream=None):
    """Gradients of delta_rule_fwd: (dq, dk, dv, dg, dbeta, dstate), dstate
    None unless wanted.  saved: what the forward call with save=True returned
    for the same inputs.  dstate_out: the gradient of state_out, where it was
    used."""
    ptrs, sizes, code, bcode = _delta_args(q, k, v, g, beta)
    Hk, Hv, dk, dv = sizes
    dt, dev = q.dtype, q.device
    if do.shape != v.shape:
        raise ValueError(f"do has shape {tuple(do.shape)}, v {tuple(v.shape)}")
    T, N, cu = _packing(v.shape[:-2], cu_seqlens, dev)
    dop, dos = _tokens(do, "do", 2, dt, dev)
    dso = _dense(dstate_out, "dstate_out", (N, Hv, dk, dv), torch.float32, dev)
    savedp = _dense(saved, "saved", saved.shape, torch.uint8, dev)
    scale = dk ** -0.5 if scale is None else scale
    with _on(stream, dev):
        dq = torch.empty(q.shape, dtype=dt, device=dev)
        dk_ = torch.empty(k.shape, dtype=dt, device=dev)
        dv_ = torch.empty(v.shape, dtype=dt, device=dev)
        dg = torch.empty(g.shape, dtype=torch.float32, device=dev)
        db = torch.empty(beta.shape, dtype=beta.dtype, device=dev)
        ds = torch.empty((N, Hv, dk, dv), dtype=torch.float32, device=dev) if want_dstate else None
        ws = _bytes(_size("delta_rule_bwd_workspace_size", T, N, *sizes, code), dev)
        _check("delta_rule_bwd",
               _mixer_lib().delta_rule_bwd(dop, dos, dso, *ptrs, cu, savedp, saved.numel(), dq.data_ptr(),
                                           dk_.data_ptr(), dv_.data_ptr(), dg.data_ptr(), db.data_ptr(), _ptr(ds), T,
                                           N, *sizes, scale, qk_norm, code, bcode, _raw(stream, dev), _ptr(ws),
                                           ws.numel() if ws is not None else 0))
    return dq, dk_, dv_, dg, db, ds


def delta_rule_step(q, k, v, g, beta, pool, slots=None, *, scale=None, qk_norm=False, out=None, stream=None):
    """One token, or a few, for each request: o [R, Hv, dv] from q, k
    [R, Hk, dk], v [R, Hv, dv], g, beta [R, Hv], or all of them with a token
    axis [R, L, ...] (taken one after another); the requests' states
    pool[slots] ([P, Hv, dk, dv] fp32) are updated in place.  slots as for
    conv1d_causal_step."""
    ptrs, sizes, code, bcode = _delta_args(q, k, v, g, beta)
    Hk, Hv, dk, dv = sizes
    R, L = v.shape[0], v.shape[1] if v.dim() == 4 else 1
    dev = q.device
    if pool.dim() != 4:
        raise ValueError("pool is [P, Hv, dk, dv]")
    P = pool.shape[0]
    pp = _dense(pool, "pool", (P, Hv, dk, dv), torch.float32, dev)
    sp = _dense(slots, "slots", (R,), torch.int32, dev)
    with _on(stream, dev):
        o = torch.empty(v.shape, dtype=q.dtype, device=dev) if out is None else out
        _check("delta_rule_step",
               _mixer_lib().delta_rule_step(*ptrs, pp, sp, _dense(o, "out", v.shape, q.dtype, dev), R, L, P, *sizes,
                                            dk ** -0.5 if scale is None else scale, qk_norm, code, bcode,
                                            _raw(stream, dev)))
    return o


# ------------------------------------------------------------------- branch norm


def _norm_args(x, y, w_post, gate, w_next, act):
    if y.dim() < 1:
        raise ValueError("y is [..., D]")
    D, dt, dev = y.shape[-1], y.dtype, y.device
    code = _code(y, "y")
    R = y.numel() // D if D else 0
    if gate is not None:
        if gate.dim() < 1 or gate.shape[-1] != D:
            raise ValueError(f"gate has shape {tuple(gate.shape)}: rows of {D} wanted")
        G = gate.numel() // D if D else 0
        if R and (G < 1 or R % G):
            raise ValueError(f"{G} gate rows do not divide {R} rows")
        gp = _dense(gate, "gate", gate.shape, dt, dev)
    else:
        G, gp = max(R, 1), None
    ptrs = (_dense(x, "x", y.shape, dt, dev), _dense(y, "y", y.shape, dt, dev), _dense(w_post, "w_post", (D,), dt, dev),
            gp, _dense(w_next, "w_next", (D,), dt, dev))
    return ptrs, R, D, G, code, _act(act, ("none", "silu", "sigmoid"))


def branch_norm_fwd(x, y, w_post, gate=None, w_next=None, *, alpha=1.0, eps=1e-6, act="none", save=False, stream=None):
    """The end of a block; returns (r, h, stats).

        u = y / rms(y) * w_post;  r = x + alpha * act(gate) * u;  h = r / rms(r) * w_next

    y: [..., D], the branch; x: the residual stream, or None (nothing is
    added); gate: [..., D] with as many rows as y, one, or a number that
    divides them (consecutive rows then share one); w_next: the next block's
    norm, or None (h is None).  stats (save): what branch_norm_bwd takes."""
    ptrs, R, D, G, code, a = _norm_args(x, y, w_post, gate, w_next, act)
    dev = y.device
    with _on(stream, dev):
        r = torch.empty(y.shape, dtype=y.dtype, device=dev)
        h = torch.empty(y.shape, dtype=y.dtype, device=dev) if w_next is not None else None
        stats = torch.empty((2, R), dtype=torch.float32, device=dev) if save else None
        _check("branch_norm_fwd",
               _mixer_lib().branch_norm_fwd(*ptrs, r.data_ptr(), _ptr(h), _ptr(stats), R, D, G, alpha, eps, a, code,
                                            _raw(stream, dev)))
    return r, h, stats


def branch_norm_bwd(dr, dh, x, y, w_post, gate, w_next, stats, *, alpha=1.0, eps=1e-6, act="none", stream=None):
    """Gradients of branch_norm_fwd: (dx, dy, dw_post, dgate, dw_next), None
    for absent inputs.  dr, dh: gradients of r and h, None for zero."""
    ptrs, R, D, G, code, a = _norm_args(x, y, w_post, gate, w_next, act)
    dt, dev = y.dtype, y.device
    drp, dhp = _dense(dr, "dr", y.shape, dt, dev), _dense(dh, "dh", y.shape, dt, dev)
    if dh is not None and w_next is None:
        raise ValueError("dh goes with w_next")
    sp = _dense(stats, "stats", (2, R), torch.float32, dev)
    with _on(stream, dev):
        dx, dy, dw, dgate, dwn = (None if t is None else torch.empty(t.shape, dtype=dt, device=dev)
                                  for t in (x, y, w_post, gate, w_next))
        ws = _bytes(_size("branch_norm_bwd_workspace_size", R, D, G), dev) if R else None
        _check("branch_norm_bwd",
               _mixer_lib().branch_norm_bwd(drp, dhp, *ptrs, sp, _ptr(dx), _ptr(dy), _ptr(dw), _ptr(dgate), _ptr(dwn),
                                            R, D, G, alpha, eps, a, code, _raw(stream, dev), _ptr(ws),
                                            ws.numel() if ws is not None else 0))
    return dx, dy, dw, dgate, dwn


# ------------------------------------------------------------- differentiable forms


class _Last(torch.autograd.Function):
    """A gradient, and the tensors it depends on: it has none itself."""

    @staticmethod
    def forward(ctx, g, *depends):
        return g.view_as(g)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("the mixing operators can be differentiated once only")


def differentiable_once(backward):
    """For a backward function that calls the library: under create_graph its
    gradients, which nothing records, would pass for constants; differentiated
    again, they raise.  (torch's own decorator lets those pass whose output
    gradient is a constant, as that of a sum is, and those that are asked for
    certain inputs only.)"""

    @functools.wraps(backward)
    def wrapper(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        depends = [t for t in (*ctx.saved_tensors, *grads) if t is not None and t.requires_grad]
        return tuple(None if g is None else _Last.apply(g.detach(), *depends) for g in out)

    return wrapper


class _Conv1d(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, state, cu_seqlens, act, want_state):
        ctx.save_for_backward(x, w, bias, state, cu_seqlens)
        ctx.act = act
        y, out = conv1d_causal_fwd(x, w, bias, cu_seqlens=cu_seqlens, state=state, act=act, want_state=want_state)
        return y, out

    @staticmethod
    @differentiable_once
    def backward(ctx, dy, dstate_out):
        x, w, bias, state, cu = ctx.saved_tensors
        dx, dw, db, ds = conv1d_causal_bwd(
            dy.contiguous(), x, w, bias, cu_seqlens=cu, state=state, act=ctx.act,
            dstate_out=None if dstate_out is None else dstate_out.contiguous(), want_dstate=state is not None)
        return dx, dw, db, ds, None, None, None


def conv1d_causal(x, w, bias=None, *, cu_seqlens=None, state=None, act="silu", want_state=False):
    """conv1d_causal_fwd as an autograd function; returns (y, state_out)."""
    return _Conv1d.apply(x, w, bias, state, cu_seqlens, act, want_state)


class _DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, state, cu_seqlens, scale, qk_norm, want_state):
        o, out, saved = delta_rule_fwd(q, k, v, g, beta, cu_seqlens=cu_seqlens, state=state, scale=scale,
                                       qk_norm=qk_norm, want_state=want_state, save=any(ctx.needs_input_grad))
        # (the state is not needed, but what depends on it is to be known)
        ctx.save_for_backward(q, k, v, g, beta, cu_seqlens, saved, state if ctx.needs_input_grad[5] else None)
        ctx.more = (scale, qk_norm, state is not None)
        return o, out

    @staticmethod
    @differentiable_once
    def backward(ctx, do, dstate_out):
        q, k, v, g, beta, cu, saved, _ = ctx.saved_tensors
        scale, qk_norm, has_state = ctx.more
        grads = delta_rule_bwd(do.contiguous(), q, k, v, g, beta, saved, cu_seqlens=cu, scale=scale, qk_norm=qk_norm,
                               dstate_out=None if dstate_out is None else dstate_out.contiguous(),
                               want_dstate=has_state)
        return (*grads, None, None, None, None)


def delta_rule(q, k, v, g, beta, *, cu_seqlens=None, state=None, scale=None, qk_norm=False, want_state=False):
    """delta_rule_fwd as an autograd function; returns (o, state_out)."""
    return _DeltaRule.apply(q, k, v, g, beta, state, cu_seqlens, scale, qk_norm, want_state)


class _BranchNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, w_post, gate, w_next, alpha, eps, act):
        r, h, stats = branch_norm_fwd(x, y, w_post, gate, w_next, alpha=alpha, eps=eps, act=act,
                                      save=any(ctx.needs_input_grad))
        ctx.save_for_backward(x, y, w_post, gate, w_next, stats)
        ctx.more = {"alpha": alpha, "eps": eps, "act": act}
        ctx.set_materialize_grads(False)
        return r, h

    @staticmethod
    @differentiable_once
    def backward(ctx, dr, dh):
        x, y, w_post, gate, w_next, stats = ctx.saved_tensors
        dr, dh = (None if t is None else t.contiguous() for t in (dr, dh))
        grads = branch_norm_bwd(dr, dh, x, y, w_post, gate, w_next, stats, **ctx.more)
        return (*grads, None, None, None)


def branch_norm(x, y, w_post, gate=None, w_next=None, *, alpha=1.0, eps=1e-6, act="none"):
    """branch_norm_fwd as an autograd function; returns (r, h)."""
    return _BranchNorm.apply(x, y, w_post, gate, w_next, alpha, eps, act)
