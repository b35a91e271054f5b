"""A state space block and the TTT layer on the token grid of images or video, prefill,
decoding and training:

    u        = N(x)                                     ttt_block_norm_fwd
    c, z     = u Win
    v        = silu(conv(c))                            ttt_short_conv_fwd
    r, B, C  = v Wx
    y        = scan(v, r Wdt; A, B, C, D) silu(z)       ttt_selective_scan_fwd
    h, w     = x + y Wout, N(h)                         ttt_block_norm_fwd
    q, k     = rope(w Wq, w Wk) at (time, height, width)   ttt_rope_axes
    out      = h + TTT-Linear(q, k, w Wv) Wo            ttt_linear_fwd

The state space half is trained through the operators' backward passes; the TTT layer's own
outer gradient is not part of this library, so the second half is used as it is.

    python examples/state_space_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from test_sequence_layers_gb300 import abi, rotary  # noqa: E402


class ShortConv(torch.autograd.Function):
    """The short convolution from zero states, differentiable; reset marks where packed
    sequences begin."""

    @staticmethod
    def forward(ctx, x, weight, bias, reset):
        y, _ = abi.ttt_short_conv_fwd(x, weight, bias, reset=reset)
        ctx.save_for_backward(x, weight, bias, reset)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, reset = ctx.saved_tensors
        g = abi.ttt_short_conv_bwd(dy.contiguous(), x, weight, bias, reset=reset)
        return g.x, g.weight, g.bias, None


class SelectiveScan(torch.autograd.Function):
    """The selective scan from zero states, differentiable."""

    @staticmethod
    def forward(ctx, x, delta, A, B, C, D, z, delta_bias, reset):
        y, _, states = abi.ttt_selective_scan_fwd(x, delta, A, B, C, D=D, z=z, delta_bias=delta_bias, reset=reset,
                                                  want_states=True)
        ctx.save_for_backward(x, delta, A, B, C, D, z, delta_bias, reset, states)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, delta, A, B, C, D, z, delta_bias, reset, states = ctx.saved_tensors
        g = abi.ttt_selective_scan_bwd(dy.contiguous(), x, delta, A, B, C, states, D=D, z=z, delta_bias=delta_bias, reset=reset)
        return g.x, g.delta, g.A, g.B, g.C, g.D, g.z, g.delta_bias, None


class StateSpaceBlock:
    def __init__(self, H=8, d=64, N=16, rank=32, K=4, grid=(4, 14, 14), dtype=torch.bfloat16, seed=0, device="cuda"):
        W, E = H * d, 2 * H * d
        g = torch.Generator().manual_seed(seed)
        self.H, self.d, self.W, self.E, self.N, self.rank, self.K, self.grid, self.dtype = H, d, W, E, N, rank, K, grid, dtype

        def w(*shape):
            return (torch.randn(*shape, generator=g) / shape[0] ** 0.5).to(device, dtype)

        def v(t):
            return t.float().to(device)
        self.Win, self.Wx, self.Wdt, self.Wout = w(W, 2 * E), w(E, rank + 2 * N), w(rank, E), w(E, W)
        self.conv_w, self.conv_b = v(torch.randn(E, K, generator=g) / K ** 0.5), v(torch.zeros(E))
        self.A_log = v(torch.log(torch.arange(1, N + 1).float()).expand(E, N).contiguous())
        rate = torch.exp(torch.rand(E, generator=g) * 4.6 - 6.9)  # 0.001 .. 0.1
        self.D, self.delta_bias = v(torch.ones(E)), v(torch.log(torch.expm1(rate)))
        self.norm = v(torch.ones(W))
        self.Wqkv, self.Wo = w(W, 3 * W), w(W, W)
        self.W0 = v(0.02 * torch.randn(H, d, d, generator=g))
        # a quarter of the pairs for time, the rest for height and width
        pairs = d // 2
        time = pairs - 2 * (3 * pairs // 8)
        self.axis = rotary.rope_axes((time, 3 * pairs // 8, 3 * pairs // 8))
        self.table = rotary.rope_axes_table(max(grid), self.axis, device=device)

    def parameters(self):
        """The trained ones, of the state space half."""
        return [self.Win, self.conv_w, self.conv_b, self.Wx, self.Wdt, self.A_log, self.D, self.delta_bias, self.Wout]

    def start(self, B):
        """The state of B sequences before their first token: the convolution's last inputs, the
        scan's states, the TTT layer's inner weights, the place on the grid."""
        dev = self.W0.device
        return {"conv": torch.zeros(B, self.K - 1, self.E, device=dev, dtype=self.dtype),
                "h": torch.zeros(B, self.E, self.N, device=dev), "W": self.W0.expand(B, *self.W0.shape).contiguous(), "pos": 0}

    def ttt_half(self, h, state):
        B, T, _ = h.shape
        _, w, _ = abi.ttt_block_norm_fwd(h, pre="rms", pre_weight=self.norm)
        qkv = (w @ self.Wqkv).view(B, T, 3, self.H, self.d).permute(2, 0, 3, 1, 4)
        q, k, v = abi.ttt_rope_axes(*qkv.unbind(0), self.table, self.axis, grid=self.grid, pos0=state["pos"])
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(t.dtype) for t in (q, k))
        o, _ = abi.ttt_linear_fwd(q, k, v, state["W"], 1, eta_scalar=0.5, W_out=state["W"])
        return h + o.transpose(1, 2).reshape(B, T, self.W) @ self.Wo

    def __call__(self, x, state):
        """Prefill (x [B,T,W]) or a decoding step (T = 1); steps `state` in place."""
        with torch.no_grad():
            _, u, _ = abi.ttt_block_norm_fwd(x, pre="rms", pre_weight=self.norm)
            cz = u @ self.Win
            v, _ = abi.ttt_short_conv_fwd(cz[..., :self.E], self.conv_w, self.conv_b, state=state["conv"], state_out=state["conv"])
            p = v @ self.Wx
            r, N = self.rank, self.N
            y, _, _ = abi.ttt_selective_scan_fwd(v, p[..., :r] @ self.Wdt, -self.A_log.exp(), p[..., r:r + N], p[..., r + N:],
                                                 D=self.D, z=cz[..., self.E:], delta_bias=self.delta_bias, h0=state["h"],
                                                 h_last=state["h"])
            out = self.ttt_half(x + y @ self.Wout, state)
            state["pos"] += x.shape[1]
        return out

    def train_half(self, x, reset):
        """The state space half, differentiable in parameters(); reset marks packed sequences."""
        _, u, _ = abi.ttt_block_norm_fwd(x, pre="rms", pre_weight=self.norm)
        cz = u @ self.Win
        v = ShortConv.apply(cz[..., :self.E], self.conv_w, self.conv_b, reset)
        p = v @ self.Wx
        r, N = self.rank, self.N
        y = SelectiveScan.apply(v, p[..., :r] @ self.Wdt, -self.A_log.exp(), p[..., r:r + N], p[..., r + N:], self.D,
                                cz[..., self.E:], self.delta_bias, reset)
        return x + y @ self.Wout

    def gradients(self, x, target, reset):
        """(loss, gradients of parameters()) of one training step."""
        params = [t.requires_grad_() for t in self.parameters()]
        loss = (self.train_half(x, reset).float() - target).square().mean()
        grads = torch.autograd.grad(loss, params)
        for t in params:
            t.requires_grad_(False)
        return float(loss.detach()), grads


def main():
    torch.manual_seed(0)
    B, grid = 2, (2, 6, 5)
    block = StateSpaceBlock(H=4, d=64, N=16, rank=16, grid=grid)
    T = grid[0] * grid[1] * grid[2]
    x = torch.randn(B, T, block.W, device="cuda").to(torch.bfloat16)
    whole = block(x, block.start(B))
    state, cut = block.start(B), 37
    parts = [block(x[:, :cut].contiguous(), state)] + [block(x[:, t:t + 1].contiguous(), state) for t in range(cut, T)]
    abi.ttt_sync_status()
    joined = torch.cat(parts, 1)
    err = float((joined.float() - whole.float()).abs().max() / whole.float().abs().max())
    print(f"prefill of {T} tokens against {cut} + {T - cut} decoding steps: relative difference {err:.1e}")

    reset = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    reset[:, 25] = True  # two packed sequences
    target = torch.randn(B, T, block.W, device="cuda")
    losses = []
    for _ in range(4):
        loss, grads = block.gradients(x, target, reset)
        losses.append(loss)
        for p, g in zip(block.parameters(), grads):
            p -= 0.05 * g
    print("training the state space half: loss", " ".join(f"{v:.4f}" for v in losses))
    return err, losses


if __name__ == "__main__":
    main()
