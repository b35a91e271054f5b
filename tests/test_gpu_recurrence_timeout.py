"""The recurrence's way out when a wait runs out, made to happen on the host's request and
without a GPU fault: ttt_debug_wait_limit makes each cluster's last block wait on a barrier
that nothing arrives at, for a millisecond; it leaves, the other blocks' waits for its totals
run out in turn, copies in flight land and the cluster leaves together.  The timeout is
reported and cleared, and the next call matches the token loop."""
import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import gpu_common as G
from tests.test_gpu_recurrence import _check, _inputs, _run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LIMIT_NS = 1_000_000


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,C", [(1, 4096, 64), (2, 700, 63), (1, 3000, 66), (1, 100, 64), (40, 300, 768), (3, 40000, 64)])
def test_wait_timeout_is_reported_and_the_context_stays_usable(B, T, C, dtype):
    """Clusters of several blocks and of one, one round and many, each way that rows arrive."""
    G.ensure_built()
    i = _inputs(B, T, C, "mix", dtype, resets=0.01, seed=C)
    clean = _run(i, "mix")
    _, _, states = abi.ttt_recurrence_fwd(i["x"], i["f"], i["h0"], reset=i["reset"], want_states=True)
    abi.ttt_sync_status()
    for call in (lambda: abi.ttt_recurrence_fwd(i["x"], i["f"], i["h0"], reset=i["reset"]),
                 lambda: abi.ttt_recurrence_bwd(i["dh"], i["x"], i["f"], states, reset=i["reset"])):
        abi.ttt_debug_wait_limit(LIMIT_NS)
        try:
            call()
            with pytest.raises(abi.TTTError) as e:
                abi.ttt_sync_status()
            assert e.value.code == -5
        finally:
            abi.ttt_debug_wait_limit(0)
        abi.ttt_sync_status()
        assert all(torch.equal(a, b) for a, b in zip(_run(i, "mix"), clean))
    if T < 1000:
        _check(i, "mix")
