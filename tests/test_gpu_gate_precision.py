"""Sigmoid and SiLU gates of fp32 tensors, entry by entry relative to itself.  From the
arithmetic: the exponential 2^-23, 1 + e 2^-24, its reciprocal 2^-23, two products 2^-24 each:
below 2^-21 together; the sigmoid's slope s (1 - s) has the exponential, two
reciprocals and two products, below 2^-20.  bf16 tensors: an exponential off by |g| 2^-23 of
itself (2^-17 to |g| = 64), so that the slope stored is one of the two bf16 values around the
exact one."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [768, 501, 502])
def test_sigmoid_slope(D, dtype):
    """Far from zero on both sides, where 1 - s or s alone carries it."""
    G.ensure_built()
    gate = torch.linspace(-60, 60, 40 * D).view(1, 40, D).to(dtype)
    y = torch.ones(1, 40, D, device="cuda", dtype=dtype)
    _, _, st = abi.ttt_block_norm_fwd(y, gate=gate.cuda(), act="sigmoid", want_stats=True)
    got = abi.ttt_block_norm_bwd(y, None, y, st, gate=gate.cuda(), act="sigmoid").gate.double().cpu()
    abi.ttt_sync_status()
    g = gate.double()
    want = torch.sigmoid(g) * torch.sigmoid(-g)
    if dtype == torch.float32:
        over = (got - want).abs() / (2.0 ** -20 * want)
    else:
        over = (got - want).abs() / torch.exp2(torch.floor(torch.log2(want)) - 7)
    worst = float(gate.flatten()[over.argmax()])
    assert float(over.max()) < 1, (float(over.max()), worst)
