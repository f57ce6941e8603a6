"""Timing cases of the feed-forward half of a block: the gated feed-forward
product and its gradients, the same on 8-bit and on 4-bit weights, the 4-bit
product alone, and the norm that leaves 8-bit rows for it.

`run` computes an operator either in its plain form (elementary torch
operations in float32, rounded once at the end) or, with `own` set, through
convolution_lowering_amd.ffn.  `exact` gives the same outputs from the
operators' definitions in float64.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
LEAST = 2.0 ** -100  # a row's largest value counts as this at least: its scale stays a normal number


# --------------------------------------------------------------------- cases


def listed():
    return [
        # one training step's forward and backward over a batch of full-length samples
        {"name": "ffn_train", "op": "ffn", "pass": "train", "tokens": 8192, "width": 4096, "hidden": 8192, "act": "silu",
         "dtype": "bf16"},
        # a serving batch's prompts, packed: a ragged number of tokens
        {"name": "ffn_prompts", "op": "ffn", "pass": "fwd", "tokens": 5003, "width": 4096, "hidden": 10240,
         "act": "silu", "dtype": "bf16"},
        # a large batch's generated tokens, or a short prompt
        {"name": "ffn_batch", "op": "ffn", "pass": "fwd", "tokens": 200, "width": 4096, "hidden": 10240, "act": "gelu",
         "dtype": "fp16"},
        # a few users' generated tokens: the weights are read for them alone
        {"name": "ffn_token", "op": "ffn", "pass": "fwd", "tokens": 4, "width": 4096, "hidden": 10240, "act": "silu",
         "dtype": "bf16"},
        # a small model trained in full precision, rows that fill no tile and start anywhere
        {"name": "ffn_odd_train", "op": "ffn", "pass": "train", "tokens": 333, "width": 250, "hidden": 777,
         "act": "gelu", "dtype": "fp32"},
        # prompts of a model served in 8 bits
        {"name": "ffn8_prompts", "op": "ffn8", "tokens": 8192, "width": 4096, "hidden": 10240, "act": "silu",
         "dtype": "bf16"},
        # a batch's generated tokens, 8 bits, a ragged hidden size
        {"name": "ffn8_batch", "op": "ffn8", "tokens": 61, "width": 2048, "hidden": 5000, "act": "silu",
         "dtype": "fp16"},
        # a single user's generated token: the projection back, 4 bits
        {"name": "w4_token", "op": "w4", "rows": 1, "width": 10240, "features": 4096, "group": 128, "zeros": False,
         "gated": False, "act": "none", "dtype": "bf16"},
        # a batch's generated tokens: both projections, the activation and the product, 4 bits
        {"name": "w4_batch", "op": "w4", "rows": 32, "width": 4096, "features": 10240, "group": 128, "zeros": True,
         "gated": True, "act": "silu", "dtype": "bf16"},
        # a small layer, sizes that fill no tile, small groups
        {"name": "w4_odd", "op": "w4", "rows": 7, "width": 1000, "features": 1999, "group": 32, "zeros": True,
         "gated": False, "act": "none", "dtype": "fp16"},
        # the norm before an 8-bit product over a batch of prompts: residual sum, norm, 8-bit rows
        {"name": "norm8_prompts", "op": "norm8", "rows": 16384, "width": 4096, "residual": True, "dtype": "bf16"},
        # the same for a few generated tokens: latency
        {"name": "norm8_token", "op": "norm8", "rows": 7, "width": 4000, "residual": True, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


MOST = 8192 * 4096 * 8192  # tokens x width x hidden of the largest training step


def draw(rng):
    op = rng.choice(("ffn", "ffn", "ffn8", "w4", "w4", "norm8"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    act = rng.choice(("silu", "silu", "gelu", "sigmoid"))
    if op == "ffn":
        kind = rng.choice(("fwd", "train"))
        width, hidden = _log(rng, 64, 4096), _log(rng, 64, 10240)
        if rng.random() < 0.7:  # most models' rows are whole 16-byte pieces
            width, hidden = -(-width // 8) * 8, -(-hidden // 8) * 8
        most = min(8192 if dtype != "fp32" else 2048, MOST // (width * hidden))
        return {"op": op, "pass": kind, "tokens": _log(rng, 1, most), "width": width, "hidden": hidden, "act": act,
                "dtype": dtype}
    if op == "ffn8":
        return {"op": op, "tokens": _log(rng, 1, 8192), "width": 16 * _log(rng, 4, 256), "hidden": _log(rng, 64, 10240),
                "act": act, "dtype": rng.choice(("bf16", "bf16", "fp16"))}
    if op == "w4":
        gated = rng.random() < 0.5
        return {"op": op, "rows": _log(rng, 1, 64), "width": 8 * _log(rng, 8, 1280), "features": _log(rng, 64, 10240),
                "group": rng.choice((32, 64, 128, 128)), "zeros": rng.random() < 0.5, "gated": gated,
                "act": act if gated else "none", "dtype": dtype}
    width = _log(rng, 64, 8192)
    return {"op": op, "rows": _log(rng, 1, min(16384, (1 << 26) // width)), "width": width,
            "residual": rng.random() < 0.7, "dtype": dtype}


# -------------------------------------------------------------------- inputs


def _quant8(x):
    """e4m3 rows and their scales."""
    scale = x.abs().amax(-1).clamp(min=LEAST) / E4M3_MAX
    return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), scale


def _quant4(w, group, zeros, t):
    """4-bit codes of each row's groups, two to a byte (the earlier value in
    the low half), with scales and, where wanted, zero points."""
    F, D = w.shape
    n = -(-D // group)
    parts = torch.nn.functional.pad(w, (0, n * group - D)).view(F, n, group)
    if zeros:
        lo, hi = parts.amin(-1), parts.amax(-1)
        scale = ((hi - lo).clamp(min=1e-6) / 15).to(t)
        zero = torch.round(-lo / scale.float()).to(t)
        codes = torch.round(parts / scale.float()[..., None]) + zero.float()[..., None]
    else:
        scale, zero = (parts.abs().amax(-1).clamp(min=1e-6) / 7).to(t), None
        codes = torch.round(parts / scale.float()[..., None]) + 8
    codes = codes.clamp(0, 15).to(torch.uint8).view(F, n * group)[:, :D]
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).contiguous(), scale, zero


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    s = dict(case)
    t = DTYPES[case["dtype"]]
    if case["op"] == "ffn":
        T, D, F = case["tokens"], case["width"], case["hidden"]
        s["x"] = randn(T, D).to(t)
        s["w_gate"], s["w_up"] = ((randn(F, D) * D ** -0.5).to(t) for _ in range(2))
        if case["pass"] == "train":
            s["dh"] = randn(T, F).to(t)
    elif case["op"] == "ffn8":
        T, D, F = case["tokens"], case["width"], case["hidden"]
        s["x"], s["x_scale"] = _quant8(randn(T, D))
        s["w_gate"], s["gate_scale"] = _quant8(randn(F, D) * D ** -0.5)
        s["w_up"], s["up_scale"] = _quant8(randn(F, D) * D ** -0.5)
    elif case["op"] == "w4":
        R, D, F = case["rows"], case["width"], case["features"]
        s["x"] = randn(R, D).to(t)
        s["w"] = [_quant4(randn(F, D) * D ** -0.5, case["group"], case["zeros"], t) for _ in range(1 + case["gated"])]
    else:
        R, D = case["rows"], case["width"]
        s["x"] = randn(R, D).to(t)
        s["res"] = randn(R, D).to(t) if case["residual"] else None
        s["w"] = (1 + 0.1 * randn(D)).to(t)
        s["eps"] = 1e-6
    return s


# --------------------------------------------------------------- plain forms


def _act(z, act):
    if act == "gelu":  # the tanh form
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return torch.sigmoid(z) * z if act == "silu" else torch.sigmoid(z)


def _unpack4(w, scale, zero, D, group):
    codes = torch.stack((w & 15, w >> 4), -1).view(w.shape[0], D).float()
    at = torch.arange(D, device=DEV) // group
    return (codes - (8.0 if zero is None else zero.float()[:, at])) * scale.float()[:, at]


def _plain(s):
    t = DTYPES[s["dtype"]]
    if s["op"] == "ffn":
        train = s["pass"] == "train"
        x, wg, wu = (s[n].float().requires_grad_(train) for n in ("x", "w_gate", "w_up"))
        h = _act(x @ wg.T, s["act"]) * (x @ wu.T)
        if not train:
            return {"h": h.to(t)}
        dx, dg, du = torch.autograd.grad(h, (x, wg, wu), s["dh"].float())
        return {"h": h.detach().to(t), "dx": dx.to(t), "dw_gate": dg.to(t), "dw_up": du.to(t)}
    if s["op"] == "ffn8":
        x = s["x"].float() * s["x_scale"][:, None]
        wg, wu = s["w_gate"].float() * s["gate_scale"][:, None], s["w_up"].float() * s["up_scale"][:, None]
        return {"h": (_act(x @ wg.T, s["act"]) * (x @ wu.T)).to(t)}
    if s["op"] == "w4":
        x = s["x"].float()
        y = [x @ _unpack4(*w, s["width"], s["group"]).T for w in s["w"]]
        return {"y": (_act(y[0], s["act"]) * y[1] if s["gated"] else y[0]).to(t)}
    r = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
    h = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + s["eps"]) * s["w"].float()
    q, scale = _quant8(h)
    return {"q": q, "scale": scale, "r": None if s["res"] is None else r.to(t)}


def _own(s):
    from convolution_lowering_amd import ffn
    if s["op"] == "ffn":
        three = (s["x"], s["w_gate"], s["w_up"])
        if s["pass"] != "train":
            return {"h": ffn.gated_ffn_fwd(*three, act=s["act"])[0]}
        h, saved = ffn.gated_ffn_fwd(*three, act=s["act"], save=True)
        dx, dg, du = ffn.gated_ffn_bwd(s["dh"], *three, saved, act=s["act"])
        return {"h": h, "dx": dx, "dw_gate": dg, "dw_up": du}
    if s["op"] == "ffn8":
        return {"h": ffn.gated_ffn8_fwd(s["x"], s["x_scale"], s["w_gate"], s["gate_scale"], s["w_up"], s["up_scale"],
                                        act=s["act"], dtype=DTYPES[s["dtype"]])}
    if s["op"] == "w4":
        if s["gated"]:
            (wg, sg, zg), (wu, su, zu) = s["w"]
            return {"y": ffn.gated_ffn_w4_fwd(s["x"], wg, sg, wu, su, zg, zu, group=s["group"], act=s["act"])}
        w, scales, zeros = s["w"][0]
        return {"y": ffn.linear_w4_fwd(s["x"], w, scales, zeros, group=s["group"])}
    q, scale, r = ffn.norm_quant_fwd(s["x"], s["w"], s["res"], eps=s["eps"])
    return {"q": q, "scale": scale, "r": r}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------- work


def work(case):
    e = 4 if case["dtype"] == "fp32" else 2
    if case["op"] in ("ffn", "ffn8"):
        T, D, F = case["tokens"], case["width"], case["hidden"]
        if case["op"] == "ffn8":
            return {"bytes": T * D + 2 * F * D + T * F * e + 4 * (T + 2 * F), "flops": 4 * T * D * F}
        fwd = T * D * e + 2 * F * D * e + T * F * e
        if case["pass"] == "train":  # dh in; dx and both weights' gradients out
            return {"bytes": fwd + T * F * e + T * D * e + 2 * F * D * e, "flops": 12 * T * D * F}
        return {"bytes": fwd, "flops": 4 * T * D * F}
    if case["op"] == "w4":
        R, D, F, m = case["rows"], case["width"], case["features"], 1 + case["gated"]
        groups = -(-D // case["group"])
        return {"bytes": m * F * (D // 2 + groups * e * (1 + case["zeros"])) + R * (D + F) * e, "flops": 2 * m * R * D * F}
    R, D = case["rows"], case["width"]
    return {"bytes": R * D * (e * (1 + 2 * case["residual"]) + 1) + 4 * R + D * e, "flops": 8 * R * D}


# ---------------------------------------------------- definitions in 64 bits


def _exact_act(z, act):
    """Value and slope."""
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        p = 1 / (1 + torch.exp(-2 * c * (z + 0.044715 * z ** 3)))
        return z * p, p + z * p * (1 - p) * 2 * c * (1 + 3 * 0.044715 * z ** 2)
    p = 1 / (1 + torch.exp(-z))
    return (z * p, p + z * p * (1 - p)) if act == "silu" else (p, p * (1 - p))


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "ffn":
        x, wg, wu = s["x"].double(), s["w_gate"].double(), s["w_up"].double()
        u = x @ wu.T
        a, slope = _exact_act(x @ wg.T, s["act"])
        out = {"h": a * u}
        if s["pass"] == "train":
            dh = s["dh"].double()
            dg, du = dh * u * slope, dh * a
            out.update({"dx": dg @ wg + du @ wu, "dw_gate": dg.T @ x, "dw_up": du.T @ x})
        return out
    if s["op"] == "ffn8":
        x, wg, wu = (s[n].double() for n in ("x", "w_gate", "w_up"))
        rows = s["x_scale"].double()[:, None]
        z, u = (x @ wg.T) * rows * s["gate_scale"].double(), (x @ wu.T) * rows * s["up_scale"].double()
        return {"h": _exact_act(z, s["act"])[0] * u}
    if s["op"] == "w4":
        x, D, group = s["x"].double(), s["width"], s["group"]
        ys = []
        for w, scale, zero in s["w"]:
            wide = torch.empty(w.shape[0], D, dtype=torch.float64, device=DEV)
            wide[:, 0::2], wide[:, 1::2] = w.remainder(16), w.div(16, rounding_mode="floor")
            for i in range(scale.shape[1]):
                part = wide[:, i * group:(i + 1) * group]
                part -= 8.0 if zero is None else zero[:, i:i + 1].double()
                part *= scale[:, i:i + 1].double()
            ys.append(x @ wide.T)
        return {"y": _exact_act(ys[0], s["act"])[0] * ys[1] if s["gated"] else ys[0]}
    r = s["x"].double() + (0 if s["res"] is None else s["res"].double())
    h = r / torch.sqrt((r ** 2).sum(-1, keepdim=True) / s["width"] + s["eps"]) * s["w"].double()
    scale = h.abs().amax(-1).clamp(min=LEAST) / E4M3_MAX
    return {"q": h / scale[:, None], "scale": scale, "r": None if s["res"] is None else r}
