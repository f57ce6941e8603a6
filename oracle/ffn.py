"""The feed-forward operators from their definitions, in float64, on the CPU or
wherever the inputs lie.  Gradients come from differentiating these
definitions.  Shares no code with the HIP path."""
import math

import torch

E4M3_MAX, LEAST = 448.0, 2.0 ** -100


def act(z, name):
    if name == "none":
        return z
    if name == "gelu":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    s = 1 / (1 + torch.exp(-z))
    return z * s if name == "silu" else s


def gated_ffn(x, w_gate, w_up, name):
    """x [T, D], w_gate, w_up [F, D] -> (h, g, u)."""
    g, u = x @ w_gate.T, x @ w_up.T
    return act(g, name) * u, g, u


def weights_w4(w, scales, zeros, group):
    """The values that 4-bit codes [F, D / 2] stand for."""
    codes = torch.stack((w & 15, w >> 4), -1).flatten(1).double()
    at = torch.arange(codes.shape[1], device=w.device) // group
    return (codes - (8 if zeros is None else zeros.double()[:, at])) * scales.double()[:, at]


def norm_quant(x, res, w, eps):
    """-> (n / scale, scale, r), n / scale before it is rounded to e4m3."""
    r = x if res is None else x + res
    n = r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w
    scale = n.abs().amax(-1).clamp(min=LEAST) / E4M3_MAX
    return n / scale[..., None], scale, r
