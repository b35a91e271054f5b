"""The selective state space scan on the GPU, forward and backward, against the token loop in
64 bits, within the bounds that tests/backbone_defs.py derives."""
import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import backbone_defs as D
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _args(i):
    return (i["x"], i["delta"], i["A"], i["B"], i["C"]), dict(D=i["D"], z=i["z"], delta_bias=i["delta_bias"],
                                                              softplus=i["softplus"], reset=i["reset"])


def _run(i, **kw):
    a, k = _args(i)
    y, last, states = abi.ttt_selective_scan_fwd(*a, h0=i["h0"], want_states=i["dy"] is not None, **k, **kw)
    out = {"y": y, "h_last": last}
    if i["dy"] is not None:
        g = abi.ttt_selective_scan_bwd(i["dy"], *a, states, dh_last=i["dh_last"], **k, **kw)
        out.update(dx=g.x, ddelta=g.delta, dA=g.A, dB=g.B, dC=g.C, dD=g.D, dz=g.z, ddelta_bias=g.delta_bias, dh0=g.h0)
    return {n: v for n, v in out.items() if v is not None}


def _check(i, got=None):
    got = _run(i) if got is None else got
    ref = D.scan(i)
    for n, t in got.items():
        D.close(n, t, *ref[n])
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 3, 4, 8, 9, 16, 17, 24, 32, 33, 64])
def test_states(N, dtype):
    _check(D.scan_inputs(2, 70, 40, N, dtype=dtype, seed=N))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (2, 2, 5), (1, 8, 16), (2, 9, 17), (3, 31, 64), (1, 32, 130), (2, 33, 48),
                                   (1, 64, 33), (2, 200, 24), (1, 333, 7)])
def test_sizes(B, T, C, dtype):
    _check(D.scan_inputs(B, T, C, 16, dtype=dtype, seed=T))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G,per", [(2, 16), (3, 37), (4, 8), (5, 1), (2, 160)])
def test_groups(G, per, dtype):
    _check(D.scan_inputs(2, 75, G * per, 16, G, dtype=dtype, seed=G))


@pytest.mark.parametrize("T", [5, 100])
@pytest.mark.parametrize("kw", [dict(softplus=False), dict(gate=False), dict(skip=False), dict(state=False),
                                dict(softplus=False, gate=False, skip=False, state=False)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_options(kw, T, dtype):
    _check(D.scan_inputs(2, T, 24, 16, dtype=dtype, **kw))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [7, 100, 400])
@pytest.mark.parametrize("rate", [0.02, 0.3, 1.0])
@pytest.mark.parametrize("N", [8, 16, 20, 40])
def test_packed_sequences(T, rate, N, dtype):
    _check(D.scan_inputs(2, T, 20, N, dtype=dtype, resets=rate, seed=T))


def test_a_reset_at_every_token():
    """One each at all places of the pieces that a sequence is cut into."""
    i = D.scan_inputs(140, 140, 6, 4, dtype=F32)
    i["reset"] = torch.eye(140, dtype=torch.bool, device="cuda")
    _check(i)


def test_long_and_wide():
    i = D.scan_inputs(2, 1500, 512, 16)
    got = _check(i)
    again = _run(i)
    assert all(torch.equal(got[n], again[n]) for n in got)  # sums in a fixed order


def test_many_channels_without_pieces():
    """More warps than the GPU holds: the sequence is not cut."""
    i = D.scan_inputs(64, 40, 2048, 16, train=False)
    assert abi.ttt_selective_scan_fwd_workspace(64, 40, 2048, 16) == 0
    _check(i)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,kw", [(16, {}), (8, {}), (16, dict(gate=False, state=False)), (16, dict(resets=0.05)),
                                  (16, dict(softplus=False, skip=False))])
def test_whole_sequences(N, kw, dtype):
    """Enough channels for a block a sequence, groups with a last block that is not full, a length
    that ends inside a tile."""
    assert abi.ttt_selective_scan_fwd_workspace(24, 75, 1056, 16, 2) == 0
    assert abi.ttt_selective_scan_fwd_workspace(24, 75, 2112, 8, 2) == 0
    i = D.scan_inputs(24, 75, 1056 * 16 // N, N, 2, dtype=dtype, **kw)
    if kw.get("resets"):
        i["x"][3, 20], i["reset"][3, 21] = float("inf"), True  # seen by token 20 alone
        i["dy"][3, 20], i["dy"][3, :21] = 0, 0
        got, ref = _run(dict(i, dy=None)), D.scan(dict(i, dy=None))
        for n in ("y", "h_last"):
            ok = torch.isfinite(ref[n][0])
            D.close(n, got[n][ok], ref[n][0][ok], ref[n][1][ok])
        assert bool(torch.isfinite(got["y"][3, 21:]).all())
    else:
        _check(i)


@pytest.mark.parametrize("T", [6, 300])
def test_masked_states_may_hold_anything(T):
    """Infinities and NaN in a packed sequence reach neither the next one nor its gradients."""
    i = D.scan_inputs(1, T, 40, 16, dtype=F32)
    cut = T // 2 + 1
    i["reset"] = torch.zeros(1, T, dtype=torch.bool, device="cuda")
    i["reset"][0, cut] = True
    i["dh_last"] = None
    clean = _run(i)
    j = dict(i, x=i["x"].clone(), h0=torch.full_like(i["h0"], float("nan")))
    j["x"][0, cut - 1], j["x"][0, cut - 2] = float("inf"), float("nan")
    dirty = _run(j)
    assert torch.equal(clean["h_last"], dirty["h_last"])
    for n in ("y", "dx", "ddelta", "dB", "dC", "dz"):
        assert torch.equal(clean[n][:, cut:], dirty[n][:, cut:]), n
    assert torch.equal(clean["dh0"], dirty["dh0"])


def test_rates_from_tiny_to_large():
    i = D.scan_inputs(1, 120, 24, 16, dtype=F32, seed=3)
    i["delta"] += torch.linspace(-30, 25, 24, device="cuda")
    i["delta_bias"].zero_()
    _check(i)


@pytest.mark.parametrize("B,T,C", [(2, 7, 40), (1, 3000, 40), (8, 400, 1536), (40, 40, 2048)])
@pytest.mark.parametrize("still", ["rate", "A"])
def test_a_state_without_decay_stays_as_it_is(B, T, C, still):
    """exp(0) is one exactly: with the rate or A zero and no input, states keep their bits."""
    i = D.scan_inputs(B, T, C, 16, dtype=F32, softplus=False, train=False)
    i["B"].zero_()
    (i["delta"] if still == "rate" else i["A"]).zero_()
    assert torch.equal(_run(i)["h_last"], i["h0"])


def test_gate_far_from_zero():
    i = D.scan_inputs(1, 64, 32, 16, dtype=F32, seed=4)
    i["z"] *= torch.logspace(-2, 1.8, 32, device="cuda")
    _check(i)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slices_of_projections(dtype):
    """B and C lie in one projection behind the rates' part, x and z in another; odd offsets."""
    for rank in (48, 5):
        i = D.scan_inputs(2, 90, 48, 16, dtype=dtype)
        p = torch.full((2, 90, rank + 32), 3.0, device="cuda", dtype=dtype)
        p[..., rank:rank + 16], p[..., rank + 16:] = i["B"][:, :, 0], i["C"][:, :, 0]
        xz = torch.cat([i["x"], i["z"]], -1)
        j = dict(i, x=xz[..., :48], z=xz[..., 48:], B=p[..., rank:rank + 16].unflatten(-1, (1, 16)),
                 C=p[..., rank + 16:].unflatten(-1, (1, 16)))
        _check(j)
    # [B,T,N] without a group dimension: the same values, gradients in that shape
    a, k = _args(i)
    flat = abi.ttt_selective_scan_fwd(*a[:3], a[3][:, :, 0], a[4][:, :, 0], h0=i["h0"], want_states=True, **k)
    whole = abi.ttt_selective_scan_fwd(*a, h0=i["h0"], want_states=True, **k)
    assert all(torch.equal(s, t) for s, t in zip(flat, whole))
    g = abi.ttt_selective_scan_bwd(i["dy"], *a[:3], a[3][:, :, 0], a[4][:, :, 0], flat[2], **k)
    assert g.B.shape == (2, 90, 16) and torch.equal(g.C[:, :, None], abi.ttt_selective_scan_bwd(i["dy"], *a, flat[2], **k).C)


def test_broadcast_and_transposed_inputs():
    i = D.scan_inputs(3, 40, 16, 8, dtype=F32)
    tb = torch.empty(40, 3, 16, device="cuda").copy_(i["x"].transpose(0, 1)).transpose(0, 1)
    _check(dict(i, x=tb, B=i["B"][:1].expand(3, -1, -1, -1), dy=i["dy"][:, :1].expand(-1, 40, -1)))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unaligned_pointers(dtype):
    i = D.scan_inputs(2, 70, 32, 16, dtype=dtype)

    def off(t):
        if not isinstance(t, torch.Tensor) or t.dtype == torch.bool:
            return t
        b = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)
        b[1:].copy_(t.reshape(-1))
        return b[1:].view(t.shape)
    _check({k: off(t) for k, t in i.items()})


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [8, 16, 40])
def test_parts_and_single_tokens_in_place(N, dtype):
    """A prompt in parts, the last tokens one by one, the states stepped in place: each part's
    bound holds against the loop over the whole."""
    i = D.scan_inputs(3, 150, 24, N, dtype=dtype, resets=0.03, train=False)
    state, ys, at = i["h0"].clone(), [], 0
    for to in (70, 71, 128, *range(129, 151)):
        part = {n: (t[:, at:to].contiguous() if n in ("x", "delta", "B", "C", "z", "reset") and t is not None else t)
                for n, t in i.items()}
        a, k = _args(part)
        y, h, _ = abi.ttt_selective_scan_fwd(*a, h0=state, h_last=state, **k)
        assert h is state
        ys.append(y)
        at = to
    _check(i, {"y": torch.cat(ys, 1), "h_last": state})


def test_states_are_the_states_before_each_chunk():
    i = D.scan_inputs(2, 100, 16, 16, dtype=F32, train=False)
    a, k = _args(i)
    _, _, st = abi.ttt_selective_scan_fwd(*a, h0=i["h0"], want_states=True, **k)
    assert st.shape == (2, 4, 16, 16) and torch.equal(st[:, 0], i["h0"])
    for c in range(1, 4):
        part = {n: (t[:, :c * abi.SCAN_CHUNK] if n in ("x", "delta", "B", "C", "z") else t) for n, t in i.items()}
        D.close("states", st[:, c], *D.scan(part)["h_last"])


def test_no_tokens():
    i = D.scan_inputs(2, 0, 8, 16)
    got = _run(i)
    assert got["y"].shape == (2, 0, 8) and torch.equal(got["h_last"], i["h0"]) and torch.equal(got["dh0"], i["dh_last"])
    for n in ("dA", "dD", "ddelta_bias"):
        assert bool((got[n] == 0).all())
    i = D.scan_inputs(0, 5, 8, 16)
    assert _run(i)["dB"].shape == (0, 5, 1, 16)


def test_given_outputs_and_guards():
    i = D.scan_inputs(2, 50, 20, 12, train=False)
    a, k = _args(i)
    buf = torch.full((4, 50, 20), 7.0, device="cuda", dtype=BF)
    hb = torch.full((4, 20, 12), 7.0, device="cuda")
    sb = torch.full((4, 2, 20, 12), 7.0, device="cuda")
    y, h, st = abi.ttt_selective_scan_fwd(*a, h0=i["h0"], y=buf[1:3], h_last=hb[1:3], states=sb[1:3], **k)
    _check(i, {"y": y, "h_last": h})
    for t in (buf, hb, sb):
        assert bool((t[[0, 3]] == 7).all())


def test_gradients_along_directions():
    """The kernels' gradients against central differences of the 64-bit loop."""
    i = D.scan_inputs(1, 40, 6, 5, 2, dtype=F32, seed=9)
    got = _run(i)
    ref = D.scan(i)
    f64 = {k: t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for k, t in i.items()}
    gen = torch.Generator(device="cuda").manual_seed(5)
    for n in ("x", "delta", "A", "B", "C", "D", "z", "delta_bias", "h0"):
        v, eps, vals = torch.randn(f64[n].shape, device="cuda", dtype=torch.float64, generator=gen), 1e-5, []
        for sign in (1, -1):
            o = D.scan(dict(f64, **{n: f64[n] + sign * eps * v}))
            vals.append(float((o["y"][0] * f64["dy"]).sum() + (o["h_last"][0] * f64["dh_last"]).sum()))
        slope = (vals[0] - vals[1]) / (2 * eps)
        name = {"h0": "dh0"}.get(n, "d" + n)
        slack = float((D.bound(ref[name][0], F32, ref[name][1]) * v.abs()).sum())
        # eps^2 of the third derivative and 2^-52 of the values over eps
        assert abs(slope - float((got[name].double() * v).sum())) <= slack + 1e-7 * (1 + abs(slope)), n
