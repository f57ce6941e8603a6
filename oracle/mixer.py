"""The sequence-mixing operators from their definitions, in float64 and token
by token, on the CPU or wherever the inputs lie.  Gradients come from
differentiating these definitions.  Shares no code with the HIP path."""
import torch

DELTA_EPS = 1e-6


def _parts(cu, T):
    cu = [0, T] if cu is None else [int(c) for c in cu]
    return list(zip(cu[:-1], cu[1:]))


def conv1d_causal(x, w, bias, cu, state, act):
    """x [T, D], w [D, W], state [N, W-1, D] or None -> (y, state_out)."""
    T, D = x.shape
    W = w.shape[1]
    ys, outs = [], []
    for n, (a, e) in enumerate(_parts(cu, T)):
        head = x.new_zeros(W - 1, D) if state is None else state[n]
        line = torch.cat((head, x[a:e]))
        z = x.new_zeros(e - a, D) if bias is None else bias.expand(e - a, D)
        for j in range(W):
            z = z + line[j:j + e - a] * w[:, j]
        ys.append(z / (1 + torch.exp(-z)) if act == "silu" else z)
        outs.append(line[line.shape[0] - (W - 1):] if W > 1 else line[:0])
    return torch.cat(ys), torch.stack(outs)


def delta_rule(q, k, v, g, beta, cu, state, scale, qk_norm):
    """q, k [T, Hk, dk], v [T, Hv, dv], g, beta [T, Hv], state
    [N, Hv, dk, dv] or None -> (o, state_out)."""
    T, Hv, dv = v.shape
    rep = Hv // q.shape[1]
    if qk_norm:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + DELTA_EPS)
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + DELTA_EPS)
    q, k = q.repeat_interleave(rep, 1) * scale, k.repeat_interleave(rep, 1)
    os, outs = [], []
    for n, (a, e) in enumerate(_parts(cu, T)):
        S = v.new_zeros(Hv, q.shape[2], dv) if state is None else state[n]
        for t in range(a, e):
            S = S * torch.exp(g[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, k[t]))
            S = S + k[t][:, :, None] * u[:, None, :]
            os.append(torch.einsum("hkv,hk->hv", S, q[t]))
        outs.append(S)
    return (torch.stack(os) if os else v.new_zeros(0, Hv, dv)), torch.stack(outs)


def branch_norm(x, y, w_post, gate, w_next, alpha, eps, act):
    """y [R, D], gate [G, D] or None -> (r, h)."""
    R = y.shape[0]
    u = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w_post
    if gate is not None:
        gate = gate.repeat_interleave(R // gate.shape[0], 0)
        s = 1 / (1 + torch.exp(-gate))
        u = u * {"none": gate, "silu": gate * s, "sigmoid": s}[act]
    r = alpha * u if x is None else x + alpha * u
    if w_next is None:
        return r, None
    return r, r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w_next
