"""Feed-forward operators: the gated product with its gradients, the same on
8-bit and on 4-bit weights, the 4-bit product alone, and the norm that leaves
8-bit rows, over the C ABI of ``include/convlower_ffn.h``.

    gated_ffn_fwd / _bwd     h = act(x w_gate') * (x w_up')
    gated_ffn                the same, differentiable (once) by autograd
    gated_ffn8_fwd           ... of e4m3 rows and weights with scales
    gated_ffn_w4_fwd         ... of 4-bit weights with group scales, for a few tokens
    linear_w4_fwd            one such product
    norm_quant_fwd           e4m3 rows of norm(x + res) and their scales
    quantize_w4, quantize_rows   weights for them, once at loading

As in ``mixer``, Python only checks and marshals: outputs and workspaces are
allocated with torch on the stream the library launches on (`stream`, else the
current one of the tensors' device), and a failing call raises
ConvLowerError, ValueError or TypeError before anything is launched.

x is ``[T, D]`` or has any number of axes before D, at one stride of at most
``MAX_WIDTH`` values (norm_quant_fwd: dense); everything inside a token is dense,
and so are weights.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, lib
from .mixer import _bytes, _code, _dense, _on, _ptr, _raw, _tokens, differentiable_once

ACTS = {"none": 0, "silu": 1, "sigmoid": 2, "gelu": 3}
MAX_WIDTH, MAX_NORM_WIDTH = 1 << 20, 32768
GROUPS = (32, 64, 128)
E4M3 = torch.float8_e4m3fn
# Every symbol include/convlower_ffn.h declares.
EXPORTS = ("gated_ffn_saved_size", "gated_ffn_fwd", "gated_ffn_bwd_workspace_size", "gated_ffn_bwd", "gated_ffn_bwd_some",
           "gated_ffn8_fwd", "linear_w4_fwd", "gated_ffn_w4_fwd", "norm_quant_fwd")
_lib = None


def _ffn_lib():
    global _lib
    if _lib is None:
        L = lib()
        i, z, f, vp, l = ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_void_p, ctypes.c_int64
        L.gated_ffn_saved_size.argtypes = [l, i, ctypes.POINTER(z)]
        L.gated_ffn_fwd.argtypes = [vp, l] + [vp] * 4 + [z, l] + [i] * 4 + [vp]
        L.gated_ffn_bwd_workspace_size.argtypes = [l, i, i, i, ctypes.POINTER(z)]
        L.gated_ffn_bwd.argtypes = L.gated_ffn_bwd_some.argtypes = [vp, l, vp, l] + [vp] * 3 + [z] + [vp] * 3 + [l] + [i] * 4 + [vp, vp, z]
        L.gated_ffn8_fwd.argtypes = [vp, l] + [vp] * 6 + [l] + [i] * 4 + [vp]
        L.linear_w4_fwd.argtypes = [vp, l] + [vp] * 4 + [l] + [i] * 4 + [vp]
        L.gated_ffn_w4_fwd.argtypes = [vp, l] + [vp] * 7 + [l] + [i] * 5 + [vp]
        L.norm_quant_fwd.argtypes = [vp] * 6 + [l, i, f, i, vp]
        for name in EXPORTS:
            getattr(L, name).restype = i
        _lib = L
    return _lib


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act {act!r}: one of {tuple(ACTS)} wanted")
    return ACTS[act]


def _size(fn, *args):
    out = ctypes.c_size_t()
    _check(fn, getattr(_ffn_lib(), fn)(*args, ctypes.byref(out)))
    return out.value


def _rows(t, name, dtype, device):
    """Address, row stride and number of rows of a tensor whose last axis is
    one dense row; the axes before it lie at one stride."""
    if t.dim() < 1:
        raise ValueError(f"{name} is [..., D]")
    if t.is_contiguous():  # (the common case, without views: a one-token call is half checks)
        if t.dtype != dtype:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.device != device or not t.is_cuda:
            raise ValueError(f"{name} is on {t.device}, expected {device}, a GPU")
        D = t.shape[-1]
        return t.data_ptr(), D, t.numel() // D if D else 0
    if t.dim() > 2:
        try:
            t = t.view(-1, t.shape[-1])
        except RuntimeError:
            raise ValueError(f"{name}: its rows do not lie at one stride, strides are {tuple(t.stride())}") from None
    elif t.dim() == 1:
        t = t[None]
    return (*_tokens(t, name, 1, dtype, device), t.shape[0])


def _out(out, like, shape, device):
    """The result: the caller's tensor, checked, or a new one of `like`'s type."""
    if out is None:
        return like.new_empty(shape)
    _dense(out, "out", shape, like.dtype, device)
    return out


# ------------------------------------------------------------ gated product


def _ffn_args(x, w_gate, w_up):
    if w_gate.dim() != 2 or x.dim() < 1 or x.shape[-1] != w_gate.shape[1]:
        raise ValueError(f"x is [..., D], w_gate [F, D]: got {tuple(x.shape)} and {tuple(w_gate.shape)}")
    F, D = w_gate.shape
    dt, dev = x.dtype, x.device
    code = _code(x, "x")
    xp, xs, T = _rows(x, "x", dt, dev)
    return (code, xp, xs, _dense(w_gate, "w_gate", (F, D), dt, dev), _dense(w_up, "w_up", (F, D), dt, dev), T, D, F)


def gated_ffn_fwd(x, w_gate, w_up, *, act="silu", save=False, stream=None):
    """h = act(x w_gate') * (x w_up'); returns (h, saved).

    x: [..., D]; w_gate, w_up: [F, D]; h: [..., F].  act: "silu", "gelu" (its
    tanh form), "sigmoid" or "none".  save: what gated_ffn_bwd of the same call
    takes as `saved` (both products, fp32), else None."""
    code, xp, xs, gp, up, T, D, F = _ffn_args(x, w_gate, w_up)
    a, dev = _act(act), x.device
    with _on(stream, dev):
        h = x.new_empty((*x.shape[:-1], F))
        saved = _bytes(max(16, _size("gated_ffn_saved_size", T, F)), dev) if save else None
        _check("gated_ffn_fwd",
               _ffn_lib().gated_ffn_fwd(xp, xs, gp, up, h.data_ptr(), _ptr(saved), saved.numel() if save else 0, T, D, F,
                                        a, code, _raw(stream, dev)))
    return h, saved


def gated_ffn_bwd(dh, x, w_gate, w_up, saved, *, act="silu", want_dx=True, want_dw=True, stream=None):
    """Gradients of gated_ffn_fwd: (dx, dw_gate, dw_up), None for what is not
    wanted.  saved: what the forward call with save=True returned for the same
    inputs."""
    code, xp, xs, gp, up, T, D, F = _ffn_args(x, w_gate, w_up)
    a, dt, dev = _act(act), x.dtype, x.device
    if dh.shape != (*x.shape[:-1], F):
        raise ValueError(f"dh has shape {tuple(dh.shape)}, expected {(*x.shape[:-1], F)}")
    dp, ds, _ = _rows(dh, "dh", dt, dev)
    if saved is None:
        raise ValueError("saved: gated_ffn_fwd returns it with save=True")
    # (its layout goes by T and F: that of another call would be read wrongly)
    sp = _dense(saved, "saved", (max(16, _size("gated_ffn_saved_size", T, F)),), torch.uint8, dev)
    with _on(stream, dev):
        dx = torch.empty(x.shape, dtype=dt, device=dev) if want_dx else None
        dg, du = (torch.empty((F, D), dtype=dt, device=dev) if want_dw else None for _ in range(2))
        ws = _bytes(_size("gated_ffn_bwd_workspace_size", T, D, F, code), dev)
        _check("gated_ffn_bwd",
               _ffn_lib().gated_ffn_bwd_some(dp, ds, xp, xs, gp, up, sp, saved.numel(), _ptr(dx), _ptr(dg), _ptr(du), T,
                                             D, F, a, code, _raw(stream, dev), _ptr(ws),
                                             ws.numel() if ws is not None else 0))
    return dx, dg, du


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act, save):
        h, saved = gated_ffn_fwd(x, w_gate, w_up, act=act, save=save)
        ctx.save_for_backward(x, w_gate, w_up, saved)
        ctx.act = act
        return h

    @staticmethod
    @differentiable_once
    def backward(ctx, dh):
        x, w_gate, w_up, saved = ctx.saved_tensors
        want = ctx.needs_input_grad
        return (*gated_ffn_bwd(dh.contiguous(), x, w_gate, w_up, saved, act=ctx.act, want_dx=want[0],
                               want_dw=want[1] or want[2]), None, None)


def gated_ffn(x, w_gate, w_up, *, act="silu"):
    """gated_ffn_fwd as an autograd function; returns h."""
    # (inside the function needs_input_grad counts parameters under no_grad too)
    save = torch.is_grad_enabled() and any(t.requires_grad for t in (x, w_gate, w_up))
    return _GatedFfn.apply(x, w_gate, w_up, act, save)


def gated_ffn8_fwd(x, x_scale, w_gate, gate_scale, w_up, up_scale, *, act="silu", dtype=torch.bfloat16, stream=None):
    """gated_ffn_fwd of 8-bit rows and weights; returns h (dtype: bfloat16 or
    float16).

    x: float8_e4m3fn [..., D], x_scale: fp32, one for each row ([...]); w_gate,
    w_up: float8_e4m3fn [F, D], gate_scale, up_scale: fp32 [F].  A value stands
    for itself times its row's scale."""
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"dtype {dtype}: bfloat16 or float16 wanted")
    if w_gate.dim() != 2 or x.dim() < 1 or x.shape[-1] != w_gate.shape[1]:
        raise ValueError(f"x is [..., D], w_gate [F, D]: got {tuple(x.shape)} and {tuple(w_gate.shape)}")
    F, D = w_gate.shape
    dev = x.device
    xp, xs, T = _rows(x, "x", E4M3, dev)
    args = (xp, xs, _dense(x_scale, "x_scale", x.shape[:-1], torch.float32, dev),
            _dense(w_gate, "w_gate", (F, D), E4M3, dev), _dense(gate_scale, "gate_scale", (F,), torch.float32, dev),
            _dense(w_up, "w_up", (F, D), E4M3, dev), _dense(up_scale, "up_scale", (F,), torch.float32, dev))
    a = _act(act)
    with _on(stream, dev):
        h = torch.empty((*x.shape[:-1], F), dtype=dtype, device=dev)
        _check("gated_ffn8_fwd",
               _ffn_lib().gated_ffn8_fwd(*args, h.data_ptr(), T, D, F, a, _code(h, "h"), _raw(stream, dev)))
    return h


# ------------------------------------------------------------- 4-bit weights


def _w4_args(x, w, scales, zeros, group, names=("w", "scales", "zeros")):
    if group not in GROUPS:
        raise ValueError(f"group {group}: one of {GROUPS} wanted")
    if x.dim() < 1 or x.shape[-1] % 8:
        raise ValueError(f"x has shape {tuple(x.shape)}: rows of a multiple of 8 values wanted")
    D, dt, dev = x.shape[-1], x.dtype, x.device
    if w.dim() != 2:
        raise ValueError(f"{names[0]} is [F, D / 2]")
    F = w.shape[0]
    n = (F, -(-D // group))
    return (_dense(w, names[0], (F, D // 2), torch.uint8, dev), _dense(scales, names[1], n, dt, dev),
            _dense(zeros, names[2], n, dt, dev)), D, F


def linear_w4_fwd(x, w, scales, zeros=None, *, group=128, out=None, stream=None):
    """y = x w' for 4-bit weights: [..., F] from x [..., D], D a multiple of 8.

    w: uint8 [F, D / 2], the codes of two neighbours a byte, the earlier one in
    the low half; scales, zeros: x's dtype, [F, ceil(D / group)], group 32, 64
    or 128; a weight is scale * (code - zero), zeros None: 8.  Made for a few
    tokens.  A row of x with an infinity or a NaN gives NaN."""
    ptrs, D, F = _w4_args(x, w, scales, zeros, group)
    code, dev = _code(x, "x"), x.device
    xp, xs, R = _rows(x, "x", x.dtype, dev)
    shape = (*x.shape[:-1], F)
    with _on(stream, dev):
        y = _out(out, x, shape, dev)
        st = _ffn_lib().linear_w4_fwd(xp, xs, *ptrs, y.data_ptr(), R, D, F, group, code, _raw(stream, dev))
    _check("linear_w4_fwd", st)
    return y


def gated_ffn_w4_fwd(x, w_gate, gate_scales, w_up, up_scales, gate_zeros=None, up_zeros=None, *, group=128, act="silu",
                     out=None, stream=None):
    """h = act(x w_gate') * (x w_up') for 4-bit weights, as in linear_w4_fwd;
    zero points for both or for neither."""
    gate, D, F = _w4_args(x, w_gate, gate_scales, gate_zeros, group, ("w_gate", "gate_scales", "gate_zeros"))
    up, _, F2 = _w4_args(x, w_up, up_scales, up_zeros, group, ("w_up", "up_scales", "up_zeros"))
    if F2 != F:
        raise ValueError(f"w_up has {F2} rows, w_gate {F}")
    if (gate_zeros is None) != (up_zeros is None):
        raise ValueError("zero points for both weights or for neither")
    code, a, dev = _code(x, "x"), _act(act), x.device
    xp, xs, R = _rows(x, "x", x.dtype, dev)
    shape = (*x.shape[:-1], F)
    with _on(stream, dev):
        h = _out(out, x, shape, dev)
        st = _ffn_lib().gated_ffn_w4_fwd(xp, xs, *gate, *up, h.data_ptr(), R, D, F, group, a, code, _raw(stream, dev))
    _check("gated_ffn_w4_fwd", st)
    return h


def _w4_scales(s, dtype):
    """Scales of at least s, but for their rounding to `dtype`: where that is
    coarse, below the type's normal numbers, they go up."""
    info = torch.finfo(dtype)
    near = s.to(dtype).float()
    near += torch.where(near < s * (1 - info.eps), info.tiny * info.eps, 0.0)
    return torch.where(s > 0, near, torch.ones_like(near)).to(dtype)


@torch.no_grad()
def quantize_w4(w, group=128, zeros=False):
    """(codes, scales, zeros) of weights [F, D], as linear_w4_fwd takes them:
    each group's largest value to 7 (zeros None), or its range to 0..15.  For
    loading: plain torch, in float32.

    A zero point is rounded to w's dtype as well: the range is taken as much
    wider as that may move it, so that no value is off by more than half a step
    (bfloat16: a step of a 15th of the range and a 1920th of its distance from
    zero)."""
    if group not in GROUPS:
        raise ValueError(f"group {group}: one of {GROUPS} wanted")
    if w.dim() != 2 or w.shape[1] % 8:
        raise ValueError(f"w has shape {tuple(w.shape)}: rows of a multiple of 8 values wanted")
    F, D = w.shape
    n = -(-D // group)
    # (a short last group is filled up with its own last value, which changes none of its bounds)
    parts = torch.cat((w, w[:, -1:].expand(F, n * group - D)), 1).float().view(F, n, group)
    if zeros:
        lo, hi = parts.amin(-1), parts.amax(-1)
        half, mid = (hi - lo) / 2, (hi + lo) / 2
        # a zero point is about mid / scale; its rounding moves the values by eps / 2 of that many steps
        wide = half + mid.abs() * (torch.finfo(w.dtype).eps / 2)
        scales = _w4_scales(torch.where(half > 0, wide / 7.5, torch.zeros_like(wide)), w.dtype)
        # the middle to the middle of the codes; a group of one value is that value, at code 0
        zero = torch.where(half > 0, 7.5 - mid / scales.float(), -lo).to(w.dtype)
    else:
        scales, zero = _w4_scales(parts.abs().amax(-1) / 7, w.dtype), None
    codes = torch.round(parts / scales.float()[..., None] + (8.0 if zero is None else zero.float()[..., None]))
    codes = codes.clamp(0, 15).to(torch.uint8).view(F, -1)[:, :D]
    return (codes[:, 0::2] | codes[:, 1::2] << 4).contiguous(), scales, zero


# ------------------------------------------------------------------ 8-bit rows


def norm_quant_fwd(x, w, res=None, *, eps=1e-6, want_r=True, stream=None):
    """The norm before an 8-bit product; returns (q, scale, r).

        r = x + res;  n = r / rms(r) * w;  scale = max(max |n|, 2^-100) / 448;  q = n / scale

    x, res: [..., D]; w: [D]; q: float8_e4m3fn [..., D]; scale: fp32 [...]; r: x +
    res in x's dtype, None without res or where it is not wanted."""
    if x.dim() < 1:
        raise ValueError("x is [..., D]")
    shape, dt, dev = x.shape, x.dtype, x.device
    D, code = shape[-1], _code(x, "x")
    if D < 1:
        raise ValueError("rows without values")
    R = x.numel() // D
    ptrs = (_dense(x, "x", shape, dt, dev), _dense(res, "res", shape, dt, dev), _dense(w, "w", (D,), dt, dev))
    with _on(stream, dev):
        q = torch.empty_like(x, dtype=E4M3)
        scale = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        r = torch.empty_like(x) if res is not None and want_r else None
        _check("norm_quant_fwd",
               _ffn_lib().norm_quant_fwd(*ptrs, _ptr(r), q.data_ptr(), scale.data_ptr(), R, D, eps, code,
                                         _raw(stream, dev)))
    return q, scale, r


@torch.no_grad()
def quantize_rows(w):
    """(q, scale) of weights [F, D] for gated_ffn8_fwd: each row's largest value
    to 448.  For loading: plain torch, in float32."""
    scale = w.float().abs().amax(-1).clamp(min=2.0 ** -100) / 448
    return (w.float() / scale[:, None]).clamp(-448, 448).to(E4M3), scale
