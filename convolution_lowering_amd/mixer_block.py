"""One block of a recurrent language model on this package's operators:

    h -> q, k, v, z, decay and b     1x1 channels-last convolutions (conv2d_fwd)
    q, k, v -> short causal convolution -> gated delta rule
    -> norm of each head, gated by silu(z) -> 1x1 convolution
    -> norm, gate and residual sum, and the next norm
    with `ffn`, the feed-forward half:
    -> both projections, activation and product -> 1x1 convolution
    -> norm, gate and residual sum, and the next block's norm

``MixerBlock.forward`` is differentiable and takes packed sequences (prompts,
training); ``MixerBlock.step`` takes one token for each request and keeps the
requests' states in pools.  ``MixerBlock.quantize`` makes the feed-forward
weights for serving: 8 bits, which ``MixerBlock.prompts`` takes, and 4 bits,
which ``step`` then takes.  ``python -m convolution_lowering_amd.mixer_block``
runs all of it and a few training steps.
"""
from __future__ import annotations

import torch

from . import conv2d_fwd, ffn as feed_forward, mixer


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


def _capturing(t):
    return t.is_cuda and torch.cuda.is_current_stream_capturing()


def _renewed(old, new):
    """`new`, written into the tensors of `old` where those are of its shapes,
    types and device.  Both: tensors, None, or tuples of them."""
    if new is None:
        return None
    if isinstance(new, tuple):
        return tuple(map(_renewed, old if old is not None else (None,) * len(new), new))
    if old is None or (old.shape, old.dtype, old.device) != (new.shape, new.dtype, new.device):
        return new
    if old.is_inference() and not torch.is_inference_mode_enabled():  # (not to be written to)
        return new
    return old.copy_(new)


class _Copied:
    """Which weights copies were made of, and in which state."""

    def __init__(self, weights=()):
        self.weights, self.stamps = weights, self._stamps(weights)

    @staticmethod
    def _stamps(weights):
        return [(None if w.is_inference() else w._version, w.device, w.dtype) for w in weights]

    def still(self, weights):
        return (len(self.weights) == len(weights) and all(a is b for a, b in zip(self.weights, weights)) and
                self.stamps == self._stamps(weights))

    def __reduce__(self):  # a copied or loaded block counts its weights' versions anew
        return _Copied, ()


class MixerBlock(torch.nn.Module):
    """ffn: the hidden size of a feed-forward half, None for none; act: its gate."""

    def __init__(self, width=512, qk_heads=2, v_heads=4, head=64, taps=4, dtype=torch.bfloat16, device="cuda", seed=0,
                 ffn=None, act="silu"):
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
        self.ffn, self.act, self.w8, self.w4, self._copied = ffn, act, None, None, None
        if ffn:
            self.w_ffn_gate, self.w_ffn_up = weight(ffn, width, fan=width), weight(ffn, width, fan=width)
            self.w_ffn_down = weight(width, ffn, fan=ffn)
            self.n_ffn_post, self.n_ffn_next = ones(width), ones(width)
            self.ffn_gate = torch.nn.Parameter(torch.full((1, width), 0.5, device=device, dtype=dtype))

    def _inputs(self, h):
        gates = project(h, self.w_gates)
        decay, b = gates.split(self.v_heads, -1)
        decay = -torch.exp(self.a_log) * torch.nn.functional.softplus(decay.float() + self.dt_bias)
        return project(h, self.w_qkv), project(h, self.w_z), decay, torch.sigmoid(b).contiguous()

    def _heads(self, mixed):
        n = self.qk_heads * self.head
        q, k, v = mixed.split((n, n, self.v_heads * self.head), -1)
        return (q.unflatten(-1, (-1, self.head)), k.unflatten(-1, (-1, self.head)), v.unflatten(-1, (-1, self.head)))

    def _branch(self, x, o, z):
        o, _ = mixer.branch_norm(None, o.reshape(-1, self.head), self.n_head, z.reshape(-1, self.head), act="silu")
        return project(o.view(x.shape[0], -1), self.w_out)

    def _finish(self, x, o, z):
        x, h = mixer.branch_norm(x, self._branch(x, o, z), self.n_post, self.gate, self.n_next, alpha=1.0)
        if not self.ffn:
            return x, h
        return self._ffn_end(x, project(feed_forward.gated_ffn(h, self.w_ffn_gate, self.w_ffn_up, act=self.act), self.w_ffn_down))

    def _finish8(self, x, o, z):
        """_finish with the feed-forward product in 8 bits: the residual
        stream is the same to the bit, and its norm leaves 8-bit rows."""
        x, _ = mixer.branch_norm(x, self._branch(x, o, z), self.n_post, self.gate, alpha=1.0)
        q, scale, _ = feed_forward.norm_quant_fwd(x, self.n_next)
        h = feed_forward.gated_ffn8_fwd(q, scale, *self.w8, act=self.act, dtype=x.dtype)
        return self._ffn_end(x, project(h, self.w_ffn_down))

    def _finish4(self, x, o, z):
        """_finish with the feed-forward weights in 4 bits."""
        x, h = mixer.branch_norm(x, self._branch(x, o, z), self.n_post, self.gate, self.n_next, alpha=1.0)
        (gate, sg, zg), (up, su, zu), down = self.w4
        h = feed_forward.gated_ffn_w4_fwd(h, gate, sg, up, su, zg, zu, group=self.group, act=self.act)
        return self._ffn_end(x, feed_forward.linear_w4_fwd(h, *down, group=self.group))

    def _ffn_end(self, x, y):
        return mixer.branch_norm(x, y, self.n_ffn_post, self.ffn_gate, self.n_ffn_next, alpha=1.0)

    def quantize(self, group=64, bits=(8, 4)):
        """Copies of the feed-forward weights for serving: 8 bits for
        ``prompts`` (bfloat16 and float16 blocks), 4 bits with groups of
        `group` for ``step``.  bits: which of them; without 4, ``step`` stays
        with the weights themselves, which somewhere between 32 and 64 requests
        become faster than 4-bit ones.  Where the weights have changed since (a training
        step, load_state_dict, another device or type), ``prompts`` and ``step``
        make the copies again on their stream, in place where they fit, so that a captured
        ``step`` takes the new ones too; what is written past autograd's
        knowledge (``.data``) asks for a call of this."""
        if not self.ffn:
            raise ValueError("a block without a feed-forward half")
        if not set(bits) <= {8, 4} or not bits:
            raise ValueError(f"bits {bits!r}: 8, 4 or both wanted")
        w8 = w4 = None
        if 4 in bits:  # (refuses first)
            w4 = tuple(feed_forward.quantize_w4(w, group, zeros=True) for w in self._ffn_weights())
        if 8 in bits:
            w8 = (*feed_forward.quantize_rows(self.w_ffn_gate), *feed_forward.quantize_rows(self.w_ffn_up))
        self.group, self.w8, self.w4 = group, _renewed(self.w8, w8), _renewed(self.w4, w4)
        self._copied = _Copied(self._ffn_weights())

    def _ffn_weights(self):
        return self.w_ffn_gate, self.w_ffn_up, self.w_ffn_down

    def _refresh(self):
        """The copies of the weights as they are now."""
        if self._copied is None or self._copied.still(self._ffn_weights()):
            return
        if _capturing(self.w_ffn_gate):
            raise RuntimeError("the weights have changed since quantize: call it before the capture")
        self.quantize(self.group, [n for n, w in ((8, self.w8), (4, self.w4)) if w is not None])

    def forward(self, x, h, cu_seqlens=None, states=None, want_states=False):
        """x: the residual stream [T, width], h: its norm; returns the next
        ones and, with want_states, (last conv inputs, delta states) of each
        sequence.  states: those of an earlier call on the same sequences."""
        return self._sequences(x, h, cu_seqlens, states, want_states, self._finish)

    @torch.no_grad()
    def prompts(self, x, h, cu_seqlens=None, states=None, want_states=False):
        """forward with the 8-bit weights of ``quantize``."""
        if self.w8 is None:
            raise ValueError("no 8-bit weights: call quantize first")
        self._refresh()
        return self._sequences(x, h, cu_seqlens, states, want_states, self._finish8)

    def _sequences(self, x, h, cu_seqlens, states, want_states, finish):
        qkv, z, decay, b = self._inputs(h)
        conv0, delta0 = states if states is not None else (None, None)
        mixed, conv1 = mixer.conv1d_causal(qkv, self.w_conv, self.b_conv, cu_seqlens=cu_seqlens, state=conv0,
                                           want_state=want_states)
        q, k, v = self._heads(mixed)
        o, delta1 = mixer.delta_rule(q, k, v, decay, b, cu_seqlens=cu_seqlens, state=delta0, qk_norm=True,
                                     want_state=want_states)
        x, h = finish(x, o, z)
        return (x, h, (conv1, delta1)) if want_states else (x, h)

    def pools(self, slots):
        """Empty states for `slots` requests."""
        w = self.w_conv
        return (torch.zeros(slots, self.taps - 1, w.shape[0], dtype=w.dtype, device=w.device),
                torch.zeros(slots, self.v_heads, self.head, self.head, device=w.device))

    @torch.no_grad()
    def step(self, x, h, pools, slots=None):
        """One token for each request: x, h [R, width]; request r's states are
        pools[..][slots[r]], moved on in place.  The feed-forward weights are
        those of 4 bits once ``quantize`` has made them."""
        if self.w4 is not None:
            self._refresh()
        qkv, z, decay, b = self._inputs(h)
        mixed = mixer.conv1d_causal_step(qkv, self.w_conv, self.b_conv, pools[0], slots)
        q, k, v = self._heads(mixed)
        o = mixer.delta_rule_step(q, k, v, decay, b, pools[1], slots, qk_norm=True)
        return self._finish(x, o, z) if self.w4 is None else self._finish4(x, o, z)


def _serve(block, x, cu, prompts):
    """Prompts, then four tokens each; returns the last tokens' norms."""
    h = mixer.branch_norm_fwd(None, x, block.n_next)[0]
    _, _, states = prompts(x, h, cu, want_states=True)
    pools = block.pools(8)
    slots = torch.tensor([3, 0, 6], dtype=torch.int32, device="cuda")
    for pool, state in zip(pools, states):
        pool[slots.long()] = state
    for _ in range(4):
        token = torch.randn(3, block.width, device="cuda").bfloat16()
        _, out = block.step(token, mixer.branch_norm_fwd(None, token, block.n_next)[0], pools, slots)
    return out


def _train(block, x, cu, target):
    opt = torch.optim.SGD(block.parameters(), lr=0.5)
    for i in range(5):
        _, h1 = block(x, mixer.branch_norm(None, x, block.n_next)[0], cu)
        loss = (h1.float() - target.float()).pow(2).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        print(f"training step {i}: loss {loss.item():.4f}")


def main():
    torch.manual_seed(0)
    block = MixerBlock()
    lens = [37, 200, 5]
    cu = torch.tensor([0, 37, 237, 242], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), block.width, device="cuda").bfloat16()
    with torch.no_grad():
        out = _serve(block, x, cu, block)
    print(f"prompts of {lens} tokens, then 4 tokens each: rms {out.float().pow(2).mean().sqrt().item():.4f}")
    target = torch.randn_like(x)
    _train(block, x, cu, target)
    block = MixerBlock(ffn=1536)
    print("with a feed-forward half")
    _train(block, x, cu, target)
    block.quantize()
    out = _serve(block, x, cu, block.prompts)
    print(f"prompts in 8 bits, tokens in 4: rms {out.float().pow(2).mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
