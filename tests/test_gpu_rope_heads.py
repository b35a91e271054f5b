"""More heads than a grid has rows of blocks, at a single token."""
import pytest
import torch

from test_sequence_layers_gb300 import abi, rotary
from tests import gpu_common as G

pytestmark = pytest.mark.gpu


def test_many_heads():
    G.ensure_built()
    H, d, at = 70001, 4, 3
    q = torch.randn(1, H, 1, d, device="cuda")
    table = rotary.rope_table(8, d)
    got = abi.ttt_rope(q, q, None, table, pos0=at)
    abi.ttt_sync_status()
    a, b = q.double().split(d // 2, -1)
    c, s = table[at].double().unbind(-1)
    want = torch.cat([a * c - b * s, a * s + b * c], -1)
    # two products and a sum in fp32
    bound = 2.0 ** -22 * torch.cat([a.abs() + b.abs()] * 2, -1)
    for t in got[:2]:
        assert bool(((t.double() - want).abs() <= bound).all())
