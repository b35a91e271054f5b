"""Element offsets past 32 bits: tensors of more than 2^31 elements, their last rows against
the same rows worked on by themselves."""
import pytest
import torch

from test_sequence_layers_gb300 import abi, rotary
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _room():
    G.ensure_built()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def test_rope():
    T, H, d = (1 << 20) + 77, 32, 64
    table = rotary.rope_table(256, d)
    q = torch.randn(1, T, H, d, device="cuda", dtype=BF)
    out = abi.ttt_rope(q.transpose(1, 2), None, None, table, period=256)[0]
    tail = 300
    want = abi.ttt_rope(q[:, -tail:].transpose(1, 2), None, None, table, pos0=T - tail, period=256)[0]
    abi.ttt_sync_status()
    assert torch.equal(out[:, :, -tail:], want)


@pytest.mark.parametrize("D", [2048, 2046, 2047])
def test_block_norm(D):
    T, tail = (1 << 20) + 1027, 100
    y, x = (torch.randn(1, T, D, device="cuda", dtype=BF) for _ in range(2))
    kw = dict(post="rms", pre="layer", act="silu")
    h, u, st = abi.ttt_block_norm_fwd(y, x=x, gate=x, want_stats=True, **kw)
    g = abi.ttt_block_norm_bwd(x, y, y, st, x=x, gate=x, **kw)
    ys, xs = y[:, -tail:].contiguous(), x[:, -tail:].contiguous()
    hs, us, ss = abi.ttt_block_norm_fwd(ys, x=xs, gate=xs, want_stats=True, **kw)
    gs = abi.ttt_block_norm_bwd(xs, ys, ys, ss, x=xs, gate=xs, **kw)
    abi.ttt_sync_status()
    for a, b in ((h, hs), (u, us), (st, ss), (g.y, gs.y), (g.x, gs.x), (g.gate, gs.gate)):
        assert torch.equal(a[:, -tail:], b)


@pytest.mark.parametrize("C", [2048, 2047])
def test_recurrence(C):
    """From the stored state before the last full chunk on: the forward pass rounds the same
    steps joined in another order, the backward pass needs nothing from before."""
    T = (1 << 20) + 1027
    x, f = (torch.randn(1, T, C, device="cuda", dtype=BF) for _ in range(2))
    h, last, st = abi.ttt_recurrence_fwd(x, f, want_states=True)
    dx, df, _ = abi.ttt_recurrence_bwd(x, x, f, st)
    cut = (T - 1) // abi.RECURRENCE_CHUNK * abi.RECURRENCE_CHUNK
    xs, fs = x[:, cut:].contiguous(), f[:, cut:].contiguous()
    hs, ls, ss = abi.ttt_recurrence_fwd(xs, fs, st[:, -1].contiguous(), want_states=True)
    dxs, dfs, _ = abi.ttt_recurrence_bwd(xs, xs, fs, ss)
    abi.ttt_sync_status()
    assert float((last - ls).abs().max()) <= 2.0 ** -13
    for a, b in ((h, hs), (dx, dxs), (df, dfs)):
        assert float((a[:, cut:].float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())
