"""The short convolution, the selective scan and the positions with several axes as they are
used together: the example block, decoding and training in CUDA graphs, other streams, several
host threads, offsets past 32 bits."""
import threading

import pytest
import torch

from examples import state_space_block as S
from test_sequence_layers_gb300 import abi, rotary
from tests import backbone_defs as D
from tests import gpu_common as G
from tests.test_gpu_graph import _captured
from tests.test_gpu_streams import HOLD, _overwrite, _ready

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def test_example_runs_and_decoding_equals_the_prompt():
    """The two paths round to bf16 at the same places but run the TTT layer through other
    kernels, whose bf16 class is 2e-2."""
    err, losses = S.main()
    assert err <= G.TOL_BF16 and all(l > 0 and l == l for l in losses)


def test_example_gradients():
    """Against differentiation of the definitions in 64 bits.  A gradient passes at most eight
    matrix products and operators of fp32 with sums of up to 256 terms: 8 * 2^-15 of a tensor's
    size, in its 2-norm."""
    torch.manual_seed(3)
    B, T = 2, 45
    block = S.StateSpaceBlock(H=2, d=32, N=5, rank=7, K=3, grid=(1, 9, 5), dtype=F32)
    x, target = torch.randn(B, T, block.W, device="cuda"), torch.randn(B, T, block.W, device="cuda")
    reset = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    reset[0, 20], reset[1, 44] = True, True
    torch.backends.cuda.matmul.allow_tf32 = False
    loss, grads = block.gradients(x, target, reset)
    p = [t.double().requires_grad_() for t in block.parameters()]
    Win, cw, cb, Wx, Wdt, A_log, Dv, db, Wout = p
    xd = x.double()
    u = xd / (xd.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    c, z = (u @ Win).split(block.E, -1)
    v = D.conv(dict(x=c, weight=cw, bias=cb, act="silu", reset=reset))["y"][0]
    r, Bm, Cm = (v @ Wx).split([block.rank, block.N, block.N], -1)
    y = D.scan(dict(x=v, delta=r @ Wdt, A=-A_log.exp(), B=Bm[:, :, None], C=Cm[:, :, None], D=Dv, z=z, delta_bias=db,
                    softplus=True, reset=reset))["y"][0]
    want = (xd + y @ Wout - target).square().mean()
    assert abs(loss - float(want.detach())) <= 2.0 ** -15 * loss
    for g, w in zip(grads, torch.autograd.grad(want, p)):
        assert float((g.double() - w).norm()) <= 2.0 ** -12 * float(w.norm())


def _layer(conv, scan, y1=None):
    y1, st = abi.ttt_short_conv_fwd(conv["x"], conv["weight"], conv["bias"], state=conv["state"], state_out=conv["state"])
    a = (y1, scan["delta"], scan["A"], scan["B"], scan["C"])
    y2, h, _ = abi.ttt_selective_scan_fwd(*a, D=scan["D"], z=scan["z"], delta_bias=scan["delta_bias"], h0=scan["h0"],
                                          h_last=scan["h0"])
    return y1, y2, st, h


def test_decoding_step_in_a_graph():
    """States stepped in place inside the graph, inputs changed between replays."""
    B, C, N = 5, 96, 16
    conv, scan = D.conv_inputs(B, 1, C, 4, train=False), D.scan_inputs(B, 1, C, N, train=False)
    axis = rotary.rope_axes((8, 4, 4))
    table = rotary.rope_axes_table(64, axis)
    q, pos = torch.randn(B, 3, 1, 32, device="cuda").to(BF), torch.zeros(3, B, 1, dtype=torch.int64, device="cuda")
    got = {}

    def step():
        got["out"] = [*_layer(conv, scan), abi.ttt_rope_axes(q, None, None, table, axis, positions=pos)[0]]
        pos.add_(1)
    g = _captured(step)
    inside = got["out"]
    start = [conv["state"].clone(), scan["h0"].clone()]
    tokens = [[torch.randn_like(conv["x"]), torch.randn_like(scan["delta"]), torch.randn_like(q)] for _ in range(12)]

    def go(run, outs):
        conv["state"].copy_(start[0]), scan["h0"].copy_(start[1]), pos.zero_()
        seen = []
        for new in tokens:
            for t, v in zip((conv["x"], scan["delta"], q), new):
                t.copy_(v)
            run()
            seen.append([t.clone() for t in outs()])
        abi.ttt_sync_status()
        return seen
    replayed = go(g.replay, lambda: inside)
    for a, b in zip(replayed, go(step, lambda: got["out"])):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def _train(conv, scan):
    kw = dict(reset=conv["reset"])
    y1, _ = abi.ttt_short_conv_fwd(conv["x"], conv["weight"], conv["bias"], state=conv["state"], **kw)
    k2 = dict(D=scan["D"], z=scan["z"], delta_bias=scan["delta_bias"], **kw)
    a = (y1, scan["delta"], scan["A"], scan["B"], scan["C"])
    y2, h, st = abi.ttt_selective_scan_fwd(*a, h0=scan["h0"], want_states=True, **k2)
    g2 = abi.ttt_selective_scan_bwd(scan["dy"], *a, st, dh_last=scan["dh_last"], **k2)
    g1 = abi.ttt_short_conv_bwd(g2.x, conv["x"], conv["weight"], conv["bias"], state=conv["state"], **kw)
    return [y1, y2, h, *g2, *g1]


def _pair(B, T, C, N=16, seed=0):
    conv = D.conv_inputs(B, T, C, 4, resets=0.02, seed=seed)
    return conv, dict(D.scan_inputs(B, T, C, N, seed=seed), reset=conv["reset"])


def test_training_together():
    conv, scan = _pair(2, 300, 72)
    got = _train(conv, scan)
    D.close("y1", got[0], *D.conv(dict(conv, dy=None))["y"])
    ref = D.scan(dict(scan, x=got[0]))
    names = ("y", "h_last", "dx", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias", "dh0")
    for n, t in zip(names, got[1:12]):
        D.close(n, t, *ref[n])
    ref = D.conv(dict(conv, dy=got[3], dstate_out=None))
    for n, t in zip(("dx", "dweight", "dbias", "dstate"), got[12:]):
        D.close(n, t, *ref[n])


def test_two_training_graphs_in_turn():
    """Two captured passes, each with workspaces of its own, replayed in turn and out of order."""
    jobs = [_pair(2, 400, 160), _pair(3, 150, 64, 40, seed=1)]
    graphs, outs = [], []
    for conv, scan in jobs:
        box = {}
        graphs.append(_captured(lambda: box.__setitem__("o", _train(conv, scan))))
        outs.append(box["o"])
    want = [_train(*j) for j in jobs]
    for order in ((0, 1), (1, 0), (0, 0, 1), (1,)):
        for t in (t for o in outs for t in o):
            t.zero_()
        for i in order:
            graphs[i].replay()
        abi.ttt_sync_status()
        for i in set(order):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))


def test_workspaces_outlive_the_call_on_another_stream():
    conv, scan = _pair(2, 500, 256)
    a, k = (scan["x"], scan["delta"], scan["A"], scan["B"], scan["C"]), dict(D=scan["D"], z=scan["z"], delta_bias=scan["delta_bias"])
    _, _, st = abi.ttt_selective_scan_fwd(*a, want_states=True, **k)
    side = torch.cuda.Stream()
    calls = (lambda **s: abi.ttt_selective_scan_fwd(*a, h0=scan["h0"], **k, **s)[:2],
             lambda **s: abi.ttt_selective_scan_bwd(scan["dy"], *a, st, **k, **s),
             lambda **s: abi.ttt_short_conv_bwd(conv["dy"], conv["x"], conv["weight"], conv["bias"], **s)[:3])
    sizes = (abi.ttt_selective_scan_fwd_workspace(2, 500, 256, 16), abi.ttt_selective_scan_bwd_workspace(2, 500, 256, 16),
             abi.ttt_short_conv_bwd_workspace(2, 500, 256, 4))
    assert min(sizes) > 0
    for call, n in zip(calls, sizes):
        want = call()
        _ready(side)
        with torch.cuda.stream(side):
            torch.cuda._sleep(HOLD)
        got = call(stream=side)
        keep = _overwrite([n])
        abi.ttt_sync_status(side)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(bool((t == 0xff).all()) for t in keep)


def test_host_threads_and_streams():
    """Passes of different sizes from several host threads, each on a stream of its own."""
    jobs = [_pair(1, 200 + 50 * i, 64, (4, 16, 30, 64)[i], seed=i) for i in range(4)]
    want = [_train(*j) for j in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    got = _train(*jobs[i])
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        bad.append(i)
        except Exception as e:  # a thread's failure is the test's
            bad.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


@pytest.fixture
def _room():
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of free device memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("C", [2048, 2047])
def test_conv_offsets_past_32_bits(C, _room):
    T, tail = (1 << 20) + 1027, 200
    x, dy = (torch.randn(1, T, C, device="cuda", dtype=BF) for _ in range(2))
    w = torch.randn(C, 4, device="cuda") / 2
    y, last = abi.ttt_short_conv_fwd(x, w, want_state=True)
    g = abi.ttt_short_conv_bwd(dy, x, w)
    xs, ds = x[:, -tail:].contiguous(), dy[:, -tail:].contiguous()
    before = x[:, -tail - 3:-tail].contiguous()
    ys, ls = abi.ttt_short_conv_fwd(xs, w, state=before, want_state=True)
    gs = abi.ttt_short_conv_bwd(ds, xs, w, state=before)
    abi.ttt_sync_status()
    assert torch.equal(y[:, -tail:], ys) and torch.equal(last, ls) and torch.equal(g.x[:, -tail:], gs.x)


def test_scan_offsets_past_32_bits(_room):
    """From the stored state before the last full chunk on: the forward and the backward pass round the
    same steps cut into other pieces."""
    T, C, N = (1 << 20) + 1027, 2048, 16
    x, z = (torch.randn(1, T, C, device="cuda", dtype=BF) for _ in range(2))
    B, Cm = torch.randn(1, T, 2 * N, device="cuda", dtype=BF).split(N, -1)
    A = -torch.rand(C, N, device="cuda") - 0.5
    delta = torch.randn(1, T, C, device="cuda", dtype=BF) - 1
    y, last, st = abi.ttt_selective_scan_fwd(x, delta, A, B, Cm, z=z, want_states=True)
    g = abi.ttt_selective_scan_bwd(z, x, delta, A, B, Cm, st, z=z)
    cut = (T - 1 - 200) // abi.SCAN_CHUNK * abi.SCAN_CHUNK
    xs, zs, ds, bs, cs = (t[:, cut:].contiguous() for t in (x, z, delta, B, Cm))
    ys, ls, ss = abi.ttt_selective_scan_fwd(xs, ds, A, bs, cs, z=zs, h0=st[:, cut // abi.SCAN_CHUNK].contiguous(), want_states=True)
    gs = abi.ttt_selective_scan_bwd(zs, xs, ds, A, bs, cs, ss, z=zs)
    abi.ttt_sync_status()
    # states remember about twenty tokens here: 2^-20 a step
    assert float((last - ls).abs().max()) <= 2.0 ** -15 * float(ls.abs().max())
    for a, b in ((y, ys), (g.x, gs.x), (g.delta, gs.delta), (g.B, gs.B), (g.C, gs.C), (g.z, gs.z)):
        assert float((a[:, cut:].float() - b.float()).abs().max()) <= 2.0 ** -7 * float(b.float().abs().max())


def test_axes_offsets_past_32_bits(_room):
    T, H, d = (1 << 20) + 77, 32, 64
    axis = rotary.rope_axes((16, 8, 8), "cyclic")
    table = rotary.rope_axes_table(1 << 17, axis)
    q = torch.randn(1, T, H, d, device="cuda", dtype=BF)
    out = abi.ttt_rope_axes(q.transpose(1, 2), None, None, table, axis, grid=(1 << 17, 3, 4))[0]
    tail = 300
    want = abi.ttt_rope_axes(q[:, -tail:].transpose(1, 2), None, None, table, axis, grid=(1 << 17, 3, 4), pos0=T - tail)[0]
    abi.ttt_sync_status()
    assert torch.equal(out[:, :, -tail:], want)
