"""A position outside the rotary table and a wait that ran out, in either order: both are
reported, the timeout first."""
import pytest
import torch

from test_sequence_layers_gb300 import abi, rotary
from tests import gpu_common as G

pytestmark = pytest.mark.gpu


def _position():
    q = torch.zeros(1, 1, 4, 16, device="cuda")
    abi.ttt_rope(q, None, None, rotary.rope_table(8, 16), positions=torch.full((4,), 9, device="cuda"))


def _timeout():
    """The layer's own test of its timeout path: a first wait that can only run out."""
    inp = G.synth.make("linear", B=1, H=2, T=64, d=64, b=16, causal=True, eta="sigmoid", seed=1)
    abi.ttt_debug_wait_limit(1_000_000)
    try:
        abi.ttt_linear_fwd(*(t.cuda() for t in (inp.q, inp.k, inp.v, inp.params["W0"])), 16, eta=inp.eta.cuda())
        torch.cuda.synchronize()
    finally:
        abi.ttt_debug_wait_limit(0)


@pytest.mark.parametrize("order", [(_position, _timeout), (_timeout, _position)])
def test_neither_hides_the_other(order):
    G.ensure_built()
    abi.ttt_sync_status()
    for f in order:
        f()
    for code in (-5, -7):
        with pytest.raises(abi.TTTError) as e:
            abi.ttt_sync_status()
        assert e.value.code == code
    abi.ttt_sync_status()
