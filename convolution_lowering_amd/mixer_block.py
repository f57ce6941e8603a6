"""One block of a recurrent language model on this package's operators:

    h -> q, k, v, z, decay and b     1x1 channels-last convolutions (conv2d_fwd)
    q, k, v -> short causal convolution -> gated delta rule
    -> norm of each head, gated by silu(z) -> 1x1 convolution
    -> norm, gate and residual sum, and the next block's norm

``MixerBlock.forward`` is differentiable and takes packed sequences (prompts,
training); ``MixerBlock.step`` takes one token for each request and keeps the
requests' states in pools.  ``python -m convolution_lowering_amd.mixer_block``
runs both and a few training steps.
"""
from __future__ import annotations

import torch

from . import conv2d_fwd, mixer


class _Project(torch.autograd.Function):
    """y = x w' as a 1x1 convolution, and both gradients as two more."""

    @staticmethod
    def forward(ctx, x, w):
        ctx.save_for_backward(x, w)
        return conv2d_fwd(x[None, None], w[:, None, None], layout="NHWC").view(x.shape[0], w.shape[0])

    @staticmethod
    @mixer.differentiable_once
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dy = dy.contiguous()
        dx = conv2d_fwd(dy[None, None], w.t().contiguous()[:, None, None], layout="NHWC").view_as(x)
        # dw' = x' dy: the tokens are the channels of an image of one row, dy as it lies
        dwt = conv2d_fwd(dy[None, :, None], x.t().contiguous()[:, :, None, None], layout="NCHW")
        return dx, dwt.view(x.shape[1], w.shape[0]).t()


def project(x, w):
    """x [T, Ci], w [Co, Ci] -> [T, Co]; differentiable."""
    return _Project.apply(x, w)


class MixerBlock(torch.nn.Module):
    def __init__(self, width=512, qk_heads=2, v_heads=4, head=64, taps=4, dtype=torch.bfloat16, device="cuda", seed=0):
        super().__init__()
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape, fan):
            return torch.nn.Parameter((torch.randn(shape, generator=g, device=device) * fan ** -0.5).to(dtype))

        def ones(n):
            return torch.nn.Parameter(torch.ones(n, device=device, dtype=dtype))

        self.width, self.qk_heads, self.v_heads, self.head, self.taps = width, qk_heads, v_heads, head, taps
        qkv, inner = (2 * qk_heads + v_heads) * head, v_heads * head
        self.w_qkv, self.w_z = weight(qkv, width, fan=width), weight(inner, width, fan=width)
        self.w_gates, self.w_out = weight(2 * v_heads, width, fan=width), weight(width, inner, fan=inner)
        self.w_conv, self.b_conv = weight(qkv, taps, fan=taps), weight(qkv, fan=1e4)
        self.n_head, self.n_post, self.n_next = ones(head), ones(width), ones(width)
        self.gate = torch.nn.Parameter(torch.full((1, width), 0.5, device=device, dtype=dtype))
        # decays -exp(a_log) softplus(.. + dt_bias), float32
        self.a_log = torch.nn.Parameter(torch.rand(v_heads, generator=g, device=device))
        self.dt_bias = torch.nn.Parameter(torch.full((v_heads,), -3.0, device=device))

    def _inputs(self, h):
        gates = project(h, self.w_gates)
        decay, b = gates.split(self.v_heads, -1)
        decay = -torch.exp(self.a_log) * torch.nn.functional.softplus(decay.float() + self.dt_bias)
        return project(h, self.w_qkv), project(h, self.w_z), decay, torch.sigmoid(b).contiguous()

    def _heads(self, mixed):
        n = self.qk_heads * self.head
        q, k, v = mixed.split((n, n, self.v_heads * self.head), -1)
        return (q.unflatten(-1, (-1, self.head)), k.unflatten(-1, (-1, self.head)), v.unflatten(-1, (-1, self.head)))

    def _finish(self, x, o, z):
        o, _ = mixer.branch_norm(None, o.reshape(-1, self.head), self.n_head, z.reshape(-1, self.head), act="silu")
        y = project(o.view(x.shape[0], -1), self.w_out)
        return mixer.branch_norm(x, y, self.n_post, self.gate, self.n_next, alpha=1.0)

    def forward(self, x, h, cu_seqlens=None, states=None, want_states=False):
        """x: the residual stream [T, width], h: its norm; returns the next
        ones and, with want_states, (last conv inputs, delta states) of each
        sequence.  states: those of an earlier call on the same sequences."""
        qkv, z, decay, b = self._inputs(h)
        conv0, delta0 = states if states is not None else (None, None)
        mixed, conv1 = mixer.conv1d_causal(qkv, self.w_conv, self.b_conv, cu_seqlens=cu_seqlens, state=conv0,
                                           want_state=want_states)
        q, k, v = self._heads(mixed)
        o, delta1 = mixer.delta_rule(q, k, v, decay, b, cu_seqlens=cu_seqlens, state=delta0, qk_norm=True,
                                     want_state=want_states)
        x, h = self._finish(x, o, z)
        return (x, h, (conv1, delta1)) if want_states else (x, h)

    def pools(self, slots):
        """Empty states for `slots` requests."""
        w = self.w_conv
        return (torch.zeros(slots, self.taps - 1, w.shape[0], dtype=w.dtype, device=w.device),
                torch.zeros(slots, self.v_heads, self.head, self.head, device=w.device))

    @torch.no_grad()
    def step(self, x, h, pools, slots=None):
        """One token for each request: x, h [R, width]; request r's states are
        pools[..][slots[r]], moved on in place."""
        qkv, z, decay, b = self._inputs(h)
        mixed = mixer.conv1d_causal_step(qkv, self.w_conv, self.b_conv, pools[0], slots)
        q, k, v = self._heads(mixed)
        o = mixer.delta_rule_step(q, k, v, decay, b, pools[1], slots, qk_norm=True)
        return self._finish(x, o, z)


def main():
    torch.manual_seed(0)
    block = MixerBlock()
    lens = [37, 200, 5]
    cu = torch.tensor([0, 37, 237, 242], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), block.width, device="cuda").bfloat16()
    with torch.no_grad():
        h = mixer.branch_norm_fwd(None, x, block.n_next)[0]
        _, _, states = block(x, h, cu, want_states=True)
        pools = block.pools(8)
        slots = torch.tensor([3, 0, 6], dtype=torch.int32, device="cuda")
        for pool, state in zip(pools, states):
            pool[slots.long()] = state
        for _ in range(4):
            token = torch.randn(3, block.width, device="cuda").bfloat16()
            _, out = block.step(token, mixer.branch_norm_fwd(None, token, block.n_next)[0], pools, slots)
    print(f"prompts of {lens} tokens, then 4 tokens each: rms {out.float().pow(2).mean().sqrt().item():.4f}")
    target = torch.randn_like(x)
    opt = torch.optim.SGD(block.parameters(), lr=0.5)
    for i in range(5):
        _, h1 = block(x, mixer.branch_norm(None, x, block.n_next)[0], cu)
        loss = (h1.float() - target.float()).pow(2).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        print(f"training step {i}: loss {loss.item():.4f}")


if __name__ == "__main__":
    main()
