"""The gated linear recurrence on the GPU, forward and backward, against the token loop in
64 bits.

Tolerances, from the arithmetic.  Decays below 1 - 2^-8 for the inputs drawn here, so an
error made at one token fades within 256; every step makes at most 4 * 2^-24 of the state
(gate, product, sum): 2^-14 of the largest state in the worst case, and as much again for
joining chunks.  Relative to a tensor's largest entry: fp32 2^-13; bf16 outputs add their
one rounding, 2^-9 of each entry: 2^-8 covers both."""
import numpy as np
import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 2.0 ** -8, F32: 2.0 ** -13}
MODES = ("decay", "sigmoid", "mix")


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _inputs(B, T, C, mode, dtype, resets=0.0, seed=0, h0=True):
    g = torch.Generator().manual_seed(seed)
    f = 2.0 + 1.5 * torch.randn(B, T, C, generator=g)
    f = f.clamp(max=5.5)  # sigmoid(5.5) = 1 - 2^-8
    if mode == "decay":
        f = torch.sigmoid(f) * (1 - 2 * torch.randint(0, 2, (B, 1, C), generator=g))  # of either sign
    i = {"x": torch.randn(B, T, C, generator=g), "f": f, "dh": torch.randn(B, T, C, generator=g)}
    i = {k: t.to(dtype).cuda() for k, t in i.items()}
    i["h0"] = torch.randn(B, C, generator=g).cuda() if h0 else None
    i["dh_last"] = torch.randn(B, C, generator=g).cuda() if h0 else None
    i["reset"] = (torch.rand(B, T, generator=g) < resets).cuda() if resets else None
    return i


def _loop(i, mode):
    """h, h_last, dx, df, dh0: the recurrence token by token in 64 bits and back."""
    d = lambda t: None if t is None else t.double().cpu().numpy()
    x, f, dh, h0, dhl = (d(i[n]) for n in ("x", "f", "dh", "h0", "dh_last"))
    B, T, C = x.shape
    a = f if mode == "decay" else 1 / (1 + np.exp(-f))
    c = 1 / (1 + np.exp(f)) if mode == "mix" else np.ones_like(f)
    live = np.ones((B, T)) if i["reset"] is None else 1.0 - i["reset"].double().cpu().numpy()
    h = np.zeros((B, C)) if h0 is None else h0
    H, P = np.empty((B, T, C)), np.empty((B, T, C))
    for t in range(T):
        P[:, t] = h * live[:, t, None]
        h = a[:, t] * P[:, t] + c[:, t] * x[:, t]
        H[:, t] = h
    r = np.zeros((B, C)) if dhl is None else dhl
    dx, df = np.empty_like(x), np.empty_like(x)
    for t in range(T - 1, -1, -1):
        s = r + (0 if dh is None else dh[:, t])
        dx[:, t] = c[:, t] * s
        da = s * (P[:, t] - (x[:, t] if mode == "mix" else 0))
        df[:, t] = da if mode == "decay" else da * a[:, t] * (1 - a[:, t])
        r = a[:, t] * s * live[:, t, None]
    return H, h, dx, df, r


def _run(i, mode, **kw):
    h, hl, st = abi.ttt_recurrence_fwd(i["x"], i["f"], i["h0"], mode=mode, reset=i["reset"], want_states=True, **kw)
    g = abi.ttt_recurrence_bwd(i["dh"], i["x"], i["f"], st, mode=mode, reset=i["reset"], dh_last=i["dh_last"], **kw)
    return (h, hl, *g)


def _check(i, mode):
    got = _run(i, mode)
    abi.ttt_sync_status()
    ref = _loop(i, mode)
    for n, a, b in zip(("h", "h_last", "dx", "df", "dh0"), got, ref):
        assert tuple(a.shape) == b.shape
        # a step's error is relative to the state, so a gradient that cancels is held to its
        # factors' size: at least one
        a, e = a.double().cpu().numpy(), TOL[a.dtype]
        assert np.isfinite(a).all()
        assert np.abs(a - b).max() <= e * max(1.0, np.abs(b).max()), (n, np.abs(a - b).max(), np.abs(b).max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("B,T,C", [(1, 1, 1), (64, 1, 768), (2, 5, 64), (1, 127, 8), (3, 128, 72), (2, 129, 64),
                                   (1, 257, 333), (2, 1000, 40), (1, 4096, 16), (2, 515, 768), (5, 300, 130)])
def test_sizes(B, T, C, mode, dtype):
    _check(_inputs(B, T, C, mode, dtype, seed=T + C), mode)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", MODES)
def test_resets(mode, dtype):
    for B, T, C, p in ((2, 700, 64, 0.02), (3, 333, 17, 0.3), (1, 2048, 128, 0.001), (2, 64, 64, 1.0)):
        _check(_inputs(B, T, C, mode, dtype, resets=p, seed=T), mode)
    i = _inputs(2, 300, 64, mode, dtype, resets=0.01, seed=9)
    i["reset"][:, 0] = True  # the start state is cut off too
    _check(i, mode)


@pytest.mark.parametrize("mode", MODES)
def test_no_start_state_and_no_gradients_from_above(mode):
    i = _inputs(2, 260, 96, mode, BF, h0=False)
    _check(i, mode)
    i = _inputs(2, 260, 96, mode, BF)
    _check(dict(i, dh=None), mode)


def test_state_before_a_reset_does_not_pass_it():
    """NaN and infinity before a reset, and in the start state, stay before it, forward and
    backward (gradients after a reset do not depend on what stands before it)."""
    for mode in MODES:
        for T, cut in ((600, 300), (40, 7), (512, 256), (3000, 1)):
            i = _inputs(1, T, 64, mode, F32, seed=T)
            i["reset"] = torch.zeros(1, T, dtype=torch.bool, device="cuda")
            i["reset"][0, cut] = True
            clean = _run(i, mode)
            j = dict(i, x=i["x"].clone(), h0=i["h0"].clone())
            j["x"][0, :cut] = float("inf")
            j["x"][0, cut // 2] = float("nan")
            j["h0"][:] = float("nan")
            got = _run(j, mode)
            abi.ttt_sync_status()
            for n in (0, 2, 3):
                assert torch.equal(got[n][0, cut:], clean[n][0, cut:]), (mode, T, n)
            assert torch.equal(got[1], clean[1])
            k = dict(i, dh=i["dh"].clone(), dh_last=i["dh_last"].clone())
            k["dh"][0, cut:] = float("nan")
            k["dh_last"][:] = float("inf")
            got = _run(k, mode)
            assert torch.equal(got[2][0, :cut], clean[2][0, :cut]) and torch.equal(got[4], clean[4])


def test_saturated_gates():
    """Logits at the type's extremes and infinities: keep the state exactly, or drop it."""
    for dtype in (BF, F32):
        x = torch.randn(1, 9, 64, device="cuda").to(dtype)
        f = torch.zeros(1, 9, 64, device="cuda", dtype=dtype)
        h0 = torch.randn(1, 64, device="cuda")
        f[:, :4] = torch.finfo(dtype).max
        f[:, 2] = float("inf")
        f[:, 5] = torch.finfo(dtype).min
        f[:, 7] = -float("inf")
        h, hl, st = abi.ttt_recurrence_fwd(x, f, h0, want_states=True)
        dx, df, dh0 = abi.ttt_recurrence_bwd(torch.ones_like(x), x, f, st)
        abi.ttt_sync_status()
        assert torch.equal(h[0, 3], h0[0].to(dtype)) and torch.equal(h[0, 5], x[0, 5]) and torch.equal(h[0, 7], x[0, 7])
        assert bool((dx[0, :4] == 0).all()) and bool((df[0, [0, 1, 2, 3, 5, 7]] == 0).all())
        assert all(bool(t.isfinite().all()) for t in (h, hl, dx, df, dh0))


def test_slow_decays_keep_their_rate():
    """Mix with rates of 2^-12 over 4096 tokens of a constant input: h = 1 - (1 - eta)^t.  A
    rate formed as 1 - a would be off by 2^-13 of itself; held to 2^-16 and the sum's
    rounding, 4096 steps of 2^-25."""
    T = 4096
    f = torch.full((1, T, 64), float(np.log(2.0 ** 12 - 1)), device="cuda")
    h, hl, _ = abi.ttt_recurrence_fwd(torch.ones(1, T, 64, device="cuda"), f)
    abi.ttt_sync_status()
    eta = 1 / (1 + np.exp(np.float64(f[0, 0, 0].item())))
    want = 1 - (1 - eta) ** np.arange(1, T + 1)
    assert np.abs(h[0, :, 0].double().cpu().numpy() / want - 1).max() <= 2.0 ** -13


@pytest.mark.parametrize("mode", MODES)
def test_gradients_against_differences(mode):
    """Central differences of the kernel's forward, step 2^-7 along random unit directions:
    the third derivative's term 2^-14 / 6 of order-one curvature, rounding 2^-22 / 2^-7."""
    i = _inputs(2, 150, 24, mode, F32, resets=0.02, seed=2)
    _, _, dx, df, dh0 = _run(i, mode)

    def objective(j):
        h, hl, _ = abi.ttt_recurrence_fwd(j["x"], j["f"], j["h0"], mode=mode, reset=j["reset"])
        return float((h.double() * i["dh"].double()).sum() + (hl.double() * i["dh_last"].double()).sum())
    gen = torch.Generator().manual_seed(1)
    for n, g in (("x", dx), ("f", df), ("h0", dh0)):
        v = torch.randn(i[n].shape, generator=gen).cuda()
        v /= v.norm()
        e = 2.0 ** -7
        hi, lo = objective({**i, n: i[n] + e * v}), objective({**i, n: i[n] - e * v})
        want, scale = float((g.double() * v.double()).sum()), float(g.double().norm())
        assert abs((hi - lo) / (2 * e) - want) <= 4e-3 * max(1.0, scale), n


def test_decoding_steps_equal_one_pass_and_states_step_in_place():
    B, T, C = 4, 20, 200
    i = _inputs(B, T, C, "mix", F32, seed=5)
    h, hl, _ = abi.ttt_recurrence_fwd(i["x"], i["f"], i["h0"])
    state = i["h0"].clone()
    for t in range(T):
        ht, s, _ = abi.ttt_recurrence_fwd(i["x"][:, t:t + 1], i["f"][:, t:t + 1], state, h_last=state)
        assert s.data_ptr() == state.data_ptr()
        assert float((ht[:, 0] - h[:, t]).abs().max()) <= 2.0 ** -21 * float(h.abs().max())
    abi.ttt_sync_status()
    assert float((state - hl).abs().max()) <= 2.0 ** -21 * float(h.abs().max())
    # a long pass over the states in place, split in two
    i = _inputs(2, 3000, 64, "mix", F32, seed=6)
    want = abi.ttt_recurrence_fwd(i["x"], i["f"], i["h0"])
    state = i["h0"].clone()
    for a, b in ((0, 1300), (1300, 3000)):
        abi.ttt_recurrence_fwd(i["x"][:, a:b], i["f"][:, a:b], state, h_last=state)
    abi.ttt_sync_status()
    assert float((state - want[1]).abs().max()) <= 2.0 ** -14 * float(want[0].abs().max())


def test_strided_inputs():
    B, T, C = 2, 333, 64
    for width, off in ((3 * C, C), (3 * C + 1, C)):  # aligned slices, then odd rows
        i = _inputs(B, T, C, "mix", BF, seed=width)
        wide = torch.randn(B, T, width, device="cuda").to(BF)
        wide[..., off:off + C] = i["f"]
        j = dict(i, f=wide[..., off:off + C], x=wide[..., :C])
        _check(j, "mix")
    j = dict(i, x=i["x"][:, :1].expand(B, T, C), f=i["f"][:1].expand(B, T, C))  # broadcast inputs
    _check(j, "mix")


def test_same_bits_every_run():
    i = _inputs(2, 5000, 128, "mix", BF, seed=3)
    a = _run(i, "mix")
    for _ in range(5):
        assert all(torch.equal(s, t) for s, t in zip(a, _run(i, "mix")))


def test_no_tokens():
    x = torch.empty(2, 0, 8, device="cuda", dtype=BF)
    h0 = torch.randn(2, 8, device="cuda")
    h, hl, st = abi.ttt_recurrence_fwd(x, x, h0, want_states=True)
    dx, df, dh0 = abi.ttt_recurrence_bwd(x, x, x, st, dh_last=h0)
    abi.ttt_sync_status()
    assert h.shape == x.shape and st.shape == (2, 0, 8) and torch.equal(hl, h0) and torch.equal(dh0, h0)
    assert bool((abi.ttt_recurrence_fwd(x, x)[1] == 0).all())


def test_long_context():
    """One long sequence at the width of a head, and the long-context layer's batch (every
    channel of it, fewer of its tokens)."""
    _check(_inputs(1, 32768, 64, "mix", BF, seed=11), "mix")
    _check(_inputs(2, 4096, 2048, "mix", BF, seed=12), "mix")


def test_on_a_side_stream():
    i = _inputs(2, 2000, 128, "mix", BF)
    want = _run(i, "mix")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = _run(i, "mix")
    abi.ttt_sync_status(st)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", [1, 3, 6, 64, 65, 129])
def test_rows_that_begin_anywhere(C, dtype):
    """Tensors that start at every element of 16 bytes between NaNs, inputs and outputs: what
    stands around them neither gets in nor is written over."""
    B, T = 2, 150
    i = _inputs(B, T, C, "mix", dtype, resets=0.02, seed=C)
    n = B * T * C

    def placed(t, off):
        flat = torch.full((n + 16,), float("nan"), device="cuda", dtype=dtype)
        if t is not None:
            flat[off:off + n] = t.flatten()
        return flat, flat[off:off + n].view(B, T, C)

    def around(flat, off):
        return torch.cat((flat[:off], flat[off + n:]))
    want = _loop(i, "mix")
    for off in range(16 // i["x"].element_size()):
        j = dict(i, **{k: placed(i[k], (off + s) % 8)[1] for s, k in enumerate(("x", "f", "dh"))})
        (hb, h), (xb, dx), (fb, df) = (placed(None, (off + s) % 8) for s in range(3))
        _, hl, st = abi.ttt_recurrence_fwd(j["x"], j["f"], j["h0"], mode="mix", reset=j["reset"], want_states=True, h=h)
        _, _, dh0 = abi.ttt_recurrence_bwd(j["dh"], j["x"], j["f"], st, mode="mix", reset=j["reset"], dh_last=j["dh_last"],
                                           dx=dx, df=df)
        abi.ttt_sync_status()
        for s, flat in enumerate((hb, xb, fb)):
            assert around(flat, (off + s) % 8).isnan().all()
        for name, a, b in zip(("h", "h_last", "dx", "df", "dh0"), (h, hl, dx, df, dh0), want):
            a, e = a.double().cpu().numpy(), TOL[a.dtype]
            assert np.isfinite(a).all(), name
            assert np.abs(a - b).max() <= e * max(1.0, np.abs(b).max()), name
