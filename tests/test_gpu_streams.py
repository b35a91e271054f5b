"""stream= on the GPU: a call's memory is neither taken from work that the current stream
has still to do nor handed out again under the call's own kernels.  Both streams are held
back for some 50 ms in turn, so that a wrong order shows."""
import pytest
import torch

from test_sequence_layers_gb300 import abi, rotary
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HOLD = 100_000_000  # clock cycles


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _ready(stream):
    stream.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()


def _overwrite(sizes):
    """Fresh buffers of these sizes on the current stream, filled at once."""
    keep = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.current_stream().synchronize()
    return keep


def _norm(B=4, T=700, D=768):
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)
    y, x, gate, dh, du = (r(B, T, D).to(BF) for _ in range(5))
    kw = dict(x=x, gate=gate, act="silu", post="layer", pre="rms", post_weight=r(D), post_bias=r(D), scale=r(D),
              pre_weight=r(D))
    return y, dh, du, kw


def test_backward_workspace_outlives_the_call():
    y, dh, du, kw = _norm()
    _, _, st = abi.ttt_block_norm_fwd(y, want_stats=True, **kw)
    want = abi.ttt_block_norm_bwd(dh, du, y, st, **kw)
    side = torch.cuda.Stream()
    _ready(side)
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    got = abi.ttt_block_norm_bwd(dh, du, y, st, stream=side, **kw)
    keep = _overwrite([abi.ttt_block_norm_bwd_workspace(*y.shape)])
    abi.ttt_sync_status(side)
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)
    assert all(bool((t == 0xff).all()) for t in keep)


def test_split_forward_workspace_outlives_the_call():
    inp = G.synth.make("linear", B=1, H=4, T=2048, d=64, b=16, causal=True, eta="sigmoid", seed=700)
    q, k, v, eta, W0 = (t.cuda() for t in (inp.q, inp.k, inp.v, inp.eta, inp.params["W0"]))
    need = abi.ttt_linear_seqpar_workspace(1, 4, 2048, 64, 16)
    assert need > 0
    want = abi.ttt_linear_fwd_seqpar(q, k, v, W0, 16, eta=eta)
    side = torch.cuda.Stream()
    _ready(side)
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    got = abi.ttt_linear_fwd_seqpar(q, k, v, W0, 16, eta=eta, stream=side)
    keep = _overwrite([need])
    abi.ttt_sync_status(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert all(bool((t == 0xff).all()) for t in keep)


def test_results_are_not_put_where_the_current_stream_still_reads():
    y, dh, du, kw = _norm()
    x, f = (torch.randn(4, 700, 768, device="cuda").to(BF) for _ in range(2))
    q, table = torch.randn(4, 12, 700, 64, device="cuda").to(BF), rotary.rope_table(700, 64)
    _, _, st = abi.ttt_block_norm_fwd(y, want_stats=True, **kw)
    _, _, states = abi.ttt_recurrence_fwd(x, f, want_states=True)
    side = torch.cuda.Stream()
    calls = (lambda: abi.ttt_rope(q, None, None, table, stream=side),
             lambda: abi.ttt_block_norm_fwd(y, stream=side, **kw),
             lambda: abi.ttt_block_norm_bwd(dh, du, y, st, stream=side, **kw),
             lambda: abi.ttt_recurrence_fwd(x, f, stream=side),
             lambda: abi.ttt_recurrence_bwd(x, x, f, states, stream=side))
    for call in calls:
        _ready(side)
        want = [t for t in call() if t is not None]
        abi.ttt_sync_status(side)
        # freed on the host, still to be read on the current stream
        held = [torch.full_like(y, 3.0) for _ in range(4)]
        torch.cuda.synchronize()
        torch.cuda._sleep(HOLD)
        copies = [t + 0 for t in held]
        del held
        got = [t for t in call() if t is not None]
        abi.ttt_sync_status(side)
        torch.cuda.synchronize()
        assert all(bool((t == 3.0).all()) for t in copies)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_dropped_inputs_are_kept():
    """Inputs that the caller drops right after the call, as temporaries of its arguments."""
    x, f = (torch.randn(4, 700, 768, device="cuda").to(BF) for _ in range(2))
    want = abi.ttt_recurrence_fwd(x, f)[0]
    side = torch.cuda.Stream()
    _ready(side)
    with torch.cuda.stream(side):
        torch.cuda._sleep(HOLD)
    a, b = x.clone(), f.clone()
    torch.cuda.current_stream().synchronize()
    got = abi.ttt_recurrence_fwd(a, b, stream=side)[0]
    del a, b
    keep = _overwrite([x.nbytes])
    abi.ttt_sync_status(side)
    assert torch.equal(got, want) and len(keep) == 3
