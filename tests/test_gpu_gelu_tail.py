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
