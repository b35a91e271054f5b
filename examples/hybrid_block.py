"""A decoder block around the TTT layer, prefill, decoding and training:

    u      = N(x)                                       (the norm before the block)
    q, k   = rope(u Wq, u Wk), v = u Wv                 ttt_rope
    z      = TTT-Linear(q, k, v; eta = gate(u))         ttt_eta_gate, ttt_linear_fwd (delta rule)
    m      = LN(z) * GELU(u Wg)                         ttt_block_norm_fwd
    h, w   = x + m Wo, N(h)                             ttt_block_norm_fwd
    r      = recurrence(w Wx, w Wf)                     ttt_recurrence_fwd
    y, u'  = h + s * SiLU(w Wr) * N(r), N(y)            ttt_block_norm_fwd

The second half (recurrence, gate, residual) is trained through the operators' backward
passes; the TTT layer's own outer gradient is not part of this library, so the first half
is used as it is.

    python examples/hybrid_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from test_sequence_layers_gb300 import abi, rotary  # noqa: E402


class BlockNorm(torch.autograd.Function):
    """h = x + scale * act(gate) * N(y), u = N(h), differentiable."""

    @staticmethod
    def forward(ctx, y, x, gate, post_weight, scale, pre_weight):
        kw = dict(post="rms", act="silu", pre="rms")
        h, u, stats = abi.ttt_block_norm_fwd(y, x=x, gate=gate, post_weight=post_weight, scale=scale,
                                             pre_weight=pre_weight, want_stats=True, **kw)
        ctx.save_for_backward(y, x, gate, post_weight, scale, pre_weight, stats)
        ctx.kw = kw
        return h, u

    @staticmethod
    def backward(ctx, dh, du):
        y, x, gate, post_weight, scale, pre_weight, stats = ctx.saved_tensors
        g = abi.ttt_block_norm_bwd(dh, du, y, stats, x=x, gate=gate, post_weight=post_weight, scale=scale,
                                   pre_weight=pre_weight, **ctx.kw)
        return g.y, g.x, g.gate, g.post_weight, g.scale, g.pre_weight


class Recurrence(torch.autograd.Function):
    """The gated linear recurrence from zero states, differentiable; reset marks where packed
    sequences begin."""

    @staticmethod
    def forward(ctx, x, f, reset):
        h, _, states = abi.ttt_recurrence_fwd(x, f, reset=reset, want_states=True)
        ctx.save_for_backward(x, f, reset, states)
        return h

    @staticmethod
    def backward(ctx, dh):
        x, f, reset, states = ctx.saved_tensors
        dx, df, _ = abi.ttt_recurrence_bwd(dh, x, f, states, reset=reset)
        return dx, df, None


class HybridBlock:
    def __init__(self, H=12, d=64, max_tokens=4096, seed=0, device="cuda"):
        D, g = H * d, torch.Generator().manual_seed(seed)
        self.H, self.d, self.D = H, d, D

        def w(*shape):
            return (torch.randn(*shape, generator=g) / shape[0] ** 0.5).to(device, torch.bfloat16)
        self.Wqkv, self.Wg, self.Wo = w(D, 3 * D), w(D, D), w(D, D)
        self.theta = w(D, H).t().contiguous()
        self.W0 = (0.02 * torch.randn(H, d, d, generator=g)).to(device)
        self.Wx, self.Wf, self.Wr = (w(D, D).requires_grad_() for _ in range(3))
        one = torch.ones(D, device=device)
        self.n0, self.n1, self.b1, self.n2 = one, one.clone(), torch.zeros_like(one), one.clone()
        self.post, self.scale, self.n3 = (t.requires_grad_() for t in (one.clone(), 0.5 * one, one.clone()))
        # half the features turn, frequencies stretched for contexts four times as long
        self.table = rotary.rope_table(max_tokens, d // 2, device=device, scaling="yarn", factor=4.0,
                                       original_rows=max_tokens // 4)

    def start(self, B):
        """The state of B sequences before their first token: positions, the inner weights
        of the TTT layer, the recurrence."""
        dev = self.W0.device
        return {"pos": torch.zeros(B, 1, dtype=torch.int64, device=dev),
                "W": self.W0.expand(B, *self.W0.shape).contiguous(),
                "h": torch.zeros(B, self.D, device=dev)}

    def ttt_half(self, x, state):
        """x + TTT, and its norm; advances the inner weights."""
        B, T, D = x.shape
        _, u, _ = abi.ttt_block_norm_fwd(x, pre="rms", pre_weight=self.n0)
        q, k, v = (u @ self.Wqkv).view(B, T, 3, self.H, self.d).permute(2, 0, 3, 1, 4).unbind(0)
        pos = state["pos"] + torch.arange(T, device=x.device)
        q, k, v = abi.ttt_rope(q, k, v, self.table, positions=pos)
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(t.dtype) for t in (q, k))
        eta = abi.ttt_eta_gate(u, self.theta)
        z, _ = abi.ttt_linear_fwd(q, k, v, state["W"], 1, eta=eta, W_out=state["W"])
        m, _, _ = abi.ttt_block_norm_fwd(z, gate=u @ self.Wg, act="gelu", post="layer", post_weight=self.n1,
                                         post_bias=self.b1)
        h, w, _ = abi.ttt_block_norm_fwd(m @ self.Wo, x=x, pre="rms", pre_weight=self.n2)
        return h, w

    def __call__(self, x, state):
        """Prefill (x [B,T,D]) or a decoding step (T = 1); steps `state` in place."""
        with torch.no_grad():
            h, w = self.ttt_half(x, state)
            r, _, _ = abi.ttt_recurrence_fwd(w @ self.Wx, w @ self.Wf, state["h"], h_last=state["h"])
            y, u, _ = abi.ttt_block_norm_fwd(r, x=h, gate=w @ self.Wr, act="silu", post="rms", post_weight=self.post,
                                             scale=self.scale, pre="rms", pre_weight=self.n3)
            state["pos"] += x.shape[1]
        return y, u

    def train_step(self, x, target, reset, lr):
        """One step on the second half's weights; returns the loss before it."""
        with torch.no_grad():
            h, w = self.ttt_half(x, self.start(x.shape[0]))
        r = Recurrence.apply(w @ self.Wx, w @ self.Wf, reset)
        _, u = BlockNorm.apply(r, h, w @ self.Wr, self.post, self.scale, self.n3)
        loss = (u.float() - target).square().mean()
        params = (self.Wx, self.Wf, self.Wr, self.post, self.scale, self.n3)
        with torch.no_grad():
            for p, g in zip(params, torch.autograd.grad(loss, params)):
                p -= lr * g
        return float(loss.detach())


def main():
    torch.manual_seed(0)
    B, T = 4, 96
    block = HybridBlock(H=4, d=64, max_tokens=1024)
    x = torch.randn(B, T, block.D, device="cuda").to(torch.bfloat16)

    whole, _ = block(x, block.start(B))
    state, steps = block.start(B), []
    first, _ = block(x[:, :T // 2], state)
    for t in range(T // 2, T):
        steps.append(block(x[:, t:t + 1].contiguous(), state)[0])
    abi.ttt_sync_status()
    joined = torch.cat([first, *steps], 1)
    err = float((joined.float() - whole.float()).abs().max() / whole.float().abs().max())
    print(f"prefill of {T} tokens against {T // 2} + {T - T // 2} decoding steps: relative difference {err:.1e}")

    reset = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    reset[:, 40] = True  # two packed sequences
    target = torch.randn(B, T, block.D, device="cuda")
    losses = [block.train_step(x, target, reset, lr=2.0) for _ in range(8)]
    print("training the recurrent half: loss", " ".join(f"{v:.4f}" for v in losses))
    return err, losses


if __name__ == "__main__":
    main()
