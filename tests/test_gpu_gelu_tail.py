"""GELU gates of bf16 tensors, every value to -13: entry by entry relative to itself, as the
output is where no residual is added.  The distribution is good to 2^-14 of itself, far
inside bf16's spacing (2^-7 to 2^-8 of a value), so what is stored is one of the two bf16
values around the exact one: the error stays below one spacing.  The slope Phi + g phi is a
sum of two such terms, which cancel around -0.75: one spacing and 2^-13 of the terms."""
import numpy as np
import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _spacing(v):
    """Distance of neighbouring bf16 values around v (eight significant bits)."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -126))) - 7)


@pytest.mark.parametrize("lo,hi", [(-6.0, -3.0), (-13.0, -6.0), (-3.0, 0.0), (0.0, 13.0)])
def test_every_gate(lo, hi):
    G.ensure_built()
    every = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF)
    e64 = every.double()
    gate = every[(e64 >= lo) & (e64 <= hi) & (e64.abs() > 1e-30)]
    n = gate.numel()
    g64 = gate.double()
    phi = torch.exp(-0.5 * g64 * g64) / np.sqrt(2 * np.pi)
    cdf = torch.special.log_ndtr(g64).exp()
    for D in (768, 501, 502):  # 16-byte rows, single elements, pairs
        rows = -(-n // D)
        gt = torch.zeros(rows * D, dtype=BF)
        gt[:n] = gate
        gt = gt.view(1, rows, D).cuda()
        y = torch.ones(1, rows, D, device="cuda", dtype=BF)
        h, _, st = abi.ttt_block_norm_fwd(y, gate=gt, act="gelu", want_stats=True)
        g = abi.ttt_block_norm_bwd(y, None, y, st, gate=gt, act="gelu")
        abi.ttt_sync_status()
        h, dg, dy = (t.flatten()[:n].double().cpu() for t in (h, g.gate, g.y))
        want, slope = g64 * cdf, cdf + g64 * phi
        for got in (h, dy):
            over = (got - want).abs() / _spacing(want)
            assert float(over.max()) < 1, (D, float(over.max()), float(g64[over.argmax()]))
        over = (dg - slope).abs() - _spacing(slope) - 2.0 ** -13 * (cdf + g64.abs() * phi)
        assert float(over.max()) < 0, (D, float(g64[over.argmax()]))


def test_parameter_gradients_see_no_bias():
    """The scale's gradient, an fp32 sum over 20000 tokens of dh act(g) with dh = 1: the
    distribution is off by 2.5e-7 at most, on either side; held to 2^-20 of the sum of |act|."""
    G.ensure_built()
    B, T, D = 2, 10000, 256
    torch.manual_seed(3)
    gate = torch.randn(B, T, D, device="cuda").to(BF)
    y = torch.ones(B, T, D, device="cuda", dtype=BF)
    scale = torch.ones(D, device="cuda")
    _, _, st = abi.ttt_block_norm_fwd(y, gate=gate, act="gelu", scale=scale, want_stats=True)
    got = abi.ttt_block_norm_bwd(y, None, y, st, gate=gate, act="gelu", scale=scale).scale
    abi.ttt_sync_status()
    g = gate.double()
    act = g * torch.special.ndtr(g)
    err = (got.double() - act.sum((0, 1))).abs() / act.abs().sum((0, 1))
    assert float(err.max()) <= 2.0 ** -20, float(err.max())


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_special_gates(dtype):
    """Infinity passes, zeros and the type's extremes give 0 or g, a NaN stays in its place."""
    G.ensure_built()
    big = torch.finfo(dtype).max
    gate = torch.tensor([float("inf"), big, -big, 0.0, -0.0, float("nan"), 1.0, -100.0], dtype=dtype, device="cuda").view(1, 1, 8)
    y = torch.ones(1, 1, 8, device="cuda", dtype=dtype)
    h, _, _ = abi.ttt_block_norm_fwd(y, gate=gate, act="gelu")
    abi.ttt_sync_status()
    h = h.flatten()
    assert h[:5].tolist() == [float("inf"), big, 0.0, 0.0, 0.0] and bool(h[5].isnan()) and float(h[7]) == 0.0
    assert abs(float(h[6]) - 0.8413447) <= 2.0 ** -8
