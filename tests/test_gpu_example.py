"""The example block: a prefill equals the same tokens taken in part by decoding steps,
and training lowers the loss.  The two paths round to bf16 at the same places but run the
TTT layer and the recurrence through other kernels, whose bf16 class is 2e-2; the block
passes it through two more norms of order-one rows, hence twice that."""
import pytest

from examples import hybrid_block
from tests import gpu_common as G

pytestmark = pytest.mark.gpu


def test_example_block():
    G.ensure_built()
    err, losses = hybrid_block.main()
    assert err <= 2 * G.TOL_BF16, err
    assert losses[-1] < losses[0] and all(a > 0 for a in losses), losses
