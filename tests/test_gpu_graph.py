"""The streaming operators in CUDA graphs: captured once with preallocated outputs, replayed
over inputs that change in place, they give the bits of plain calls.  A decoding step's
states and positions step inside the graph."""
import pytest
import torch

from test_sequence_layers_gb300 import abi, rotary
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _captured(step):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    return g


def test_decoding_step():
    B, H, d = 4, 3, 64
    D = H * d
    table = rotary.rope_table(64, d)
    qkv, x, gate, f = (torch.empty(B, 1, n, device="cuda", dtype=BF) for n in (3 * D, D, D, D))
    pos, state = torch.zeros(B, 1, dtype=torch.int64, device="cuda"), torch.zeros(B, D, device="cuda")
    w = torch.randn(D, device="cuda")
    out = [torch.empty(B, H, 1, d, device="cuda", dtype=BF) for _ in range(3)]
    r, h, u = (torch.empty(B, 1, D, device="cuda", dtype=BF) for _ in range(3))

    def step():
        abi.ttt_rope(*qkv.view(B, 1, 3, H, d).permute(2, 0, 3, 1, 4).unbind(0), table, positions=pos, q_out=out[0],
                     k_out=out[1], v_out=out[2])
        abi.ttt_recurrence_fwd(x, f, state, h=r, h_last=state)
        abi.ttt_block_norm_fwd(out[0], x=r, gate=gate, post="rms", post_weight=w, pre="rms", h=h, u=u)
        pos.add_(1)
    g = _captured(step)
    gen = torch.Generator(device="cuda").manual_seed(0)
    inputs = [[torch.randn(t.shape, device="cuda", generator=gen).to(BF) for t in (qkv, x, gate, f)] for _ in range(20)]

    def go(run):
        pos.zero_(), state.zero_()
        got = []
        for new in inputs:
            for t, v in zip((qkv, x, gate, f), new):
                t.copy_(v)
            run()
            got.append([t.clone() for t in (*out, r, h, u, state)])
        abi.ttt_sync_status()
        return got
    for a, b in zip(go(step), go(g.replay)):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_training_pass():
    B, T, D = 2, 700, 256
    x, f, dh, y, w = (torch.randn(B, T, D, device="cuda").to(BF) for _ in range(4 + 1))
    vec = torch.randn(D, device="cuda")
    got = {}

    def step():
        h, last, states = abi.ttt_recurrence_fwd(x, f, want_states=True)
        o, u, st = abi.ttt_block_norm_fwd(h, x=y, gate=w, post="layer", post_weight=vec, pre="rms", want_stats=True)
        gr = abi.ttt_block_norm_bwd(dh, u, h, st, x=y, gate=w, post="layer", post_weight=vec, pre="rms")
        got["out"] = [h, last, o, u, *(t for t in gr if t is not None), *abi.ttt_recurrence_bwd(gr.y, x, f, states)]
    g = _captured(step)
    inside = got["out"]
    for seed in range(3):
        torch.manual_seed(seed)
        for t in (x, f, dh, y, w):
            t.copy_(torch.randn(t.shape, device="cuda"))
        g.replay()
        abi.ttt_sync_status()
        replayed = [t.clone() for t in inside]
        step()
        abi.ttt_sync_status()
        assert all(torch.equal(a, b) for a, b in zip(replayed, got["out"]))


def test_capture_on_the_given_stream():
    """stream= naming the stream that is captured: outputs come from the graph's own pool."""
    x, f = (torch.randn(2, 300, 64, device="cuda").to(BF) for _ in range(2))
    side, got = torch.cuda.Stream(), {}
    side.wait_stream(torch.cuda.current_stream())
    abi.ttt_recurrence_fwd(x, f, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got["h"], got["last"], _ = abi.ttt_recurrence_fwd(x, f, stream=side)
    for seed in range(3):
        torch.manual_seed(seed)
        x.copy_(torch.randn(x.shape, device="cuda"))
        g.replay()
        abi.ttt_sync_status()
        h, last, _ = abi.ttt_recurrence_fwd(x, f)
        abi.ttt_sync_status()
        assert torch.equal(h, got["h"]) and torch.equal(last, got["last"])
