"""ttt_rope in place inside one projection buffer with fewer key heads than query heads:
every slice is rotated where it stands, and equals the copy to new tensors."""
import pytest
import torch

from test_sequence_layers_gb300 import abi, rotary
from tests import gpu_common as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hk", [(4, 1), (6, 2), (1, 1)])
def test_in_place_in_a_projection_buffer(Hq, Hk):
    G.ensure_built()
    B, T, d = 2, 37, 32
    buf = torch.randn(B, T, Hq + 2 * Hk, d, device="cuda").to(torch.bfloat16)
    q, k, v = (t.transpose(1, 2) for t in buf.split([Hq, Hk, Hk], 2))
    table = rotary.rope_table(T, d)
    want = abi.ttt_rope(q, k, v, table)
    got = abi.ttt_rope(q, k, v, table, q_out=q, k_out=k, v_out=v)
    abi.ttt_sync_status()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0].data_ptr() == buf.data_ptr()
