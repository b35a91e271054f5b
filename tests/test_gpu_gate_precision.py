"""Sigmoid and SiLU gates of fp32 tensors, entry by entry relative to itself.  From the
arithmetic: the exponential 2^-23, 1 + e 2^-24, its reciprocal 2^-23, two products 2^-24 each:
below 2^-21 together."""
import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import gpu_common as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("D", [768, 501, 502])  # 16-byte rows, single elements, pairs
def test_fp32_gates(D, act):
    G.ensure_built()
    gate = torch.linspace(-80, 80, 40 * D).view(1, 40, D)
    h, _, _ = abi.ttt_block_norm_fwd(torch.ones(1, 40, D, device="cuda"), gate=gate.cuda(), act=act)
    abi.ttt_sync_status()
    g = gate.double()
    want = torch.sigmoid(g) * (g if act == "silu" else 1)
    err = ((h.double().cpu() - want) / want).abs().flatten()
    assert float(err.max()) <= 2.0 ** -21, (float(err.max()), float(gate.flatten()[err.argmax()]))
