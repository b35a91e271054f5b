"""The short causal convolution on the GPU, forward and backward, against the definition in
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


def _run(i, **kw):
    args = dict(bias=i["bias"], act=i["act"], reset=i["reset"], state=i["state"])
    y, last = abi.ttt_short_conv_fwd(i["x"], i["weight"], want_state=True, **args, **kw)
    out = {"y": y, "state_out": last}
    if i["dy"] is not None:
        g = abi.ttt_short_conv_bwd(i["dy"], i["x"], i["weight"], dstate_out=i["dstate_out"], **args, **kw)
        out.update(dx=g.x, dweight=g.weight, dbias=g.bias, dstate=g.state)
    return {k: v for k, v in out.items() if v is not None}


def _check(i, got=None):
    got = _run(i) if got is None else got
    ref = D.conv(i)
    for n, t in got.items():
        if n == "state_out":
            assert torch.equal(t.double(), ref[n][0])
        else:
            D.close(n, t, *ref[n])
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (2, 2, 8), (3, 3, 5), (2, 5, 64), (1, 130, 24), (2, 67, 30), (2, 300, 129), (5, 9, 2)])
def test_sizes(B, T, C, K, dtype):
    _check(D.conv_inputs(B, T, C, K, dtype, seed=T + K))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kw", [dict(act="none"), dict(bias=False), dict(state=False), dict(act="none", bias=False, state=False)])
def test_options(kw, dtype):
    _check(D.conv_inputs(2, 150, 40, 4, dtype, **kw))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("rate", [0.05, 0.5, 1.0])
def test_packed_sequences(K, rate, dtype):
    _check(D.conv_inputs(2, 211, 12, K, dtype, resets=rate, seed=K))


def test_resets_at_every_place_of_a_piece():
    """One reset each at tokens around the pieces that the threads take, the last rows too."""
    i = D.conv_inputs(40, 40, 8, 4, F32)
    i["reset"] = torch.eye(40, dtype=torch.bool, device="cuda")
    _check(i)


def test_long_and_wide():
    i = D.conv_inputs(2, 3000, 768, 4, BF)
    got = _check(i)
    again = _run(i)
    assert all(torch.equal(got[n], again[n]) for n in got)  # sums in a fixed order


def test_masked_rows_may_hold_anything():
    """Infinities and NaN before a sequence's start reach neither its outputs nor its gradients."""
    i = D.conv_inputs(1, 64, 16, 4, F32, state=True)
    i["reset"] = torch.zeros(1, 64, dtype=torch.bool, device="cuda")
    i["reset"][0, [0, 30]] = True
    clean = _run(i)
    i["state"][:] = float("nan")
    i["x"][0, 29, :8], i["x"][0, 28, 8:] = float("inf"), float("nan")
    dirty = _run(i)
    assert torch.equal(clean["y"][:, 30:], dirty["y"][:, 30:]) and torch.equal(clean["dx"][:, 30:], dirty["dx"][:, 30:])
    assert torch.equal(clean["y"][:, :28], dirty["y"][:, :28])
    assert torch.equal(clean["state_out"], dirty["state_out"])
    assert bool((dirty["dstate"] == 0).all())
    # the rows that were hit: what differentiation of finite rows gives is not touched by others
    assert torch.equal(clean["dx"][:, :25], dirty["dx"][:, :25])


def test_large_arguments_of_the_activation():
    i = D.conv_inputs(1, 40, 16, 4, F32, act="silu")
    i["x"] *= torch.logspace(-3, 2.5, 40, device="cuda")[None, :, None]
    _check(i)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_inputs(dtype):
    """A slice of a wider projection, a sequence-major batch, a broadcast one, odd starts."""
    base = D.conv_inputs(3, 50, 24, 4, dtype)
    wide = torch.full((3, 50, 101), 9.0, device="cuda", dtype=dtype)
    wide[..., 33:57] = base["x"]
    _check(dict(base, x=wide[..., 33:57]))
    tb = torch.empty(50, 3, 24, device="cuda", dtype=dtype)
    tb.copy_(base["dy"].transpose(0, 1))
    _check(dict(base, dy=tb.transpose(0, 1)))
    _check(dict(base, x=base["x"][:1].expand(3, -1, -1), dy=base["dy"][:, :1].expand(-1, 50, -1)))


def test_given_outputs_and_guards():
    """Outputs between guard rows, that stay as they were."""
    i = D.conv_inputs(2, 33, 20, 4, BF, train=False)
    buf = torch.full((4, 33, 20), 7.0, device="cuda", dtype=BF)
    st = torch.full((4, 3, 20), 7.0, device="cuda", dtype=BF)
    y, last = abi.ttt_short_conv_fwd(i["x"], i["weight"], i["bias"], state=i["state"], y=buf[1:3], state_out=st[1:3])
    _check(i, {"y": y, "state_out": last})
    assert bool((buf[[0, 3]] == 7).all()) and bool((st[[0, 3]] == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_single_tokens_in_place_equal_the_prompt(K, dtype):
    """Prompt at once; in parts; token by token with the state stepped in place: the same bits."""
    i = D.conv_inputs(3, 37, 40, K, dtype, resets=0.1, train=False)
    whole = _run(i)
    for cuts in ([13, 14, 20, 37], list(range(1, 38))):
        state, at, ys = i["state"].clone(), 0, []
        for to in cuts:
            y, out = abi.ttt_short_conv_fwd(i["x"][:, at:to].contiguous(), i["weight"], i["bias"],
                                            reset=i["reset"][:, at:to].contiguous(), state=state, state_out=state)
            assert out is state
            ys.append(y)
            at = to
        assert torch.equal(torch.cat(ys, 1), whole["y"]) and torch.equal(state, whole["state_out"])


def test_in_place_state_of_a_long_prompt():
    i = D.conv_inputs(2, 5000, 64, 4, BF, train=False)
    want = _run(i)
    for _ in range(5):
        state = i["state"].clone()
        y, _ = abi.ttt_short_conv_fwd(i["x"], i["weight"], i["bias"], state=state, state_out=state)
        assert torch.equal(y, want["y"]) and torch.equal(state, want["state_out"])


def test_no_tokens():
    i = D.conv_inputs(2, 0, 8, 4, BF)
    got = _run(i)
    assert got["y"].shape == (2, 0, 8) and torch.equal(got["state_out"], i["state"])
    assert bool((got["dweight"] == 0).all()) and bool((got["dbias"] == 0).all())
    assert torch.equal(got["dstate"], i["dstate_out"])
    _, z = abi.ttt_short_conv_fwd(i["x"], i["weight"], want_state=True)
    assert bool((z == 0).all())
    assert abi.ttt_short_conv_fwd(torch.empty(0, 5, 8, device="cuda", dtype=BF), i["weight"])[0].numel() == 0


def test_unaligned_pointers():
    """Every tensor one element past 16 bytes: narrower accesses, the same values."""
    i = D.conv_inputs(2, 70, 32, 4, BF)
    want = _run(i)

    def off(t):
        if t is None or t.dtype == torch.bool:
            return t
        b = torch.empty(t.numel() + 1, device="cuda", dtype=t.dtype)
        b[1:].copy_(t.reshape(-1))
        return b[1:].view(t.shape)
    j = {k: off(t) if isinstance(t, torch.Tensor) else t for k, t in i.items()}
    got = _run(j)
    for n in ("y", "dx", "state_out", "dstate"):
        assert torch.equal(want[n], got[n]), n
    _check(j, got)
