"""Block norm, gate and residual on the GPU, forward and backward, against the formula in
64 bits (gradients by differentiating it, and by differences of the kernel's own forward).

Tolerances, from the arithmetic.  fp32 inside: a row's mean and spread are sums of D terms
joined pairwise (a few 2^-24 of their absolute sums), the activations are good to 2^-21,
so each output is within 2^-17 of the largest magnitude among the terms it is made of;
those stay below 32 for the inputs drawn here (|w| <= 1.5, |y|, |x| <= 6): relative to the
output tensor's largest entry, 64 * 2^-24 times a condition of 32 = 2^-13.  bf16 outputs
add one rounding, 2^-9 of each entry, so 2^-8 covers both.  A parameter gradient sums n
tokens in fp32: sqrt(n) * 2^-24 of its terms' size, below 2^-13 of its largest entry."""
import numpy as np
import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 2.0 ** -8, F32: 2.0 ** -13}
VEC = ("post_weight", "post_bias", "scale", "pre_weight", "pre_bias")
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _inputs(B, T, D, heads, post, act, res, scale, pre, dtype, seed=0, mean=0.2):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    i = {"y": (r(B, heads, T, D // heads) if heads > 1 else r(B, T, D)) + mean,
         "x": r(B, T, D) if res else None, "gate": 2 * r(B, T, D) if act != "none" else None,
         "dh": r(B, T, D), "du": r(B, T, D) if pre != "none" else None}
    i = {k: None if t is None else t.to(dtype).cuda() for k, t in i.items()}
    on = dict(post_weight=post != "none", post_bias=post == "layer", scale=scale, pre_weight=pre != "none",
              pre_bias=pre == "layer")
    for n in VEC:
        i[n] = ((0.1 * r(D) + (0.0 if "bias" in n else 1.0)).cuda() if on[n] else None)
    return i


def _formula(i, post, act, pre, alpha):
    """h, u, and the gradients, in 64 bits on the CPU."""
    leaf = {k: (None if t is None else t.double().cpu().requires_grad_(k not in ("dh", "du"))) for k, t in i.items()}

    def norm(kind, v, w, b):
        if kind == "none":
            return v
        if kind == "layer":
            v = v - v.mean(-1, keepdim=True)
        v = v / (v.square().mean(-1, keepdim=True) + EPS).sqrt()
        return v * (1 if w is None else w) + (0 if b is None else b)
    y = leaf["y"]
    if y.dim() == 4:
        y = y.transpose(1, 2).flatten(2)
    m = norm(post, y, leaf["post_weight"], leaf["post_bias"])
    if act != "none":
        gt = leaf["gate"]
        m = m * {"sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act](gt)
    if leaf["scale"] is not None:
        m = m * leaf["scale"]
    h = m if leaf["x"] is None else alpha * leaf["x"] + m
    u = norm(pre, h, leaf["pre_weight"], leaf["pre_bias"]) if pre != "none" else None
    obj = 0.0
    if leaf["dh"] is not None:
        obj = obj + (h * leaf["dh"]).sum()
    if u is not None:
        obj = obj + (u * leaf["du"]).sum()
    obj.backward()
    grads = {n: (None if leaf[n] is None else leaf[n].grad) for n in ("y", "x", "gate") + VEC}
    return h.detach(), None if u is None else u.detach(), grads


def _rel(got, ref):
    return G.rel_err(got.double().cpu().numpy(), ref.numpy())


def _run(i, post, act, pre, alpha=1.0):
    kw = dict(x=i["x"], gate=i["gate"], act=act, post=post, pre=pre, alpha=alpha, post_eps=EPS, pre_eps=EPS,
              **{n: i[n] for n in VEC})
    h, u, stats = abi.ttt_block_norm_fwd(i["y"], want_stats=True, **kw)
    grads = abi.ttt_block_norm_bwd(i["dh"], i["du"], i["y"], stats, **kw)
    abi.ttt_sync_status()
    return h, u, grads


def _check(i, post, act, pre, alpha=1.0):
    h, u, grads = _run(i, post, act, pre, alpha)
    hr, ur, gr = _formula(i, post, act, pre, alpha)
    tol = TOL[i["y"].dtype]
    bad = {"h": _rel(h, hr)}
    if u is not None:
        bad["u"] = _rel(u, ur)
    for n in gr:
        got = getattr(grads, n)
        assert (got is None) == (gr[n] is None), n
        if got is not None and got.numel():
            assert got.shape == gr[n].shape
            bad["d" + n] = _rel(got, gr[n])
    for n, e in bad.items():
        lim = TOL[F32] if n[1:] in VEC else tol
        assert e <= lim, (n, e, lim, bad)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,heads", [(768, 12), (768, 1), (64, 1), (2048, 32), (1, 1), (7, 1), (40, 5), (33, 3), (256, 1),
                                     (257, 1), (264, 1), (1001, 1), (4096, 1), (4104, 1), (8192, 1), (8191, 1), (60, 3),
                                     (48, 2)])
def test_widths_and_layouts(D, heads, dtype):
    _check(_inputs(2, 19, D, heads, "layer", "silu", True, True, "rms", dtype, seed=D), "layer", "silu", "rms")


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("act,res,scale", [("none", False, False), ("sigmoid", True, False), ("silu", False, True),
                                           ("gelu", True, True), ("none", True, True)])
def test_every_combination(post, act, res, scale, pre):
    for D, heads, dtype in ((96, 3, BF), (333, 1, F32), (768, 1, BF)):
        i = _inputs(3, 11, D, heads, post, act, res, scale, pre, dtype, seed=D)
        if post == "none" and act == "none" and not scale and not res and pre == "none":
            i["dh"] = i["dh"].float().to(dtype)
        _check(i, post, act, pre, alpha=0.75)


@pytest.mark.parametrize("B,T", [(1, 1), (64, 1), (1, 3), (5, 1000), (1, 4097)])
def test_lengths(B, T):
    _check(_inputs(B, T, 320, 5, "rms", "gelu", True, True, "layer", BF, seed=T), "rms", "gelu", "layer")
    _check(_inputs(B, T, 56, 1, "layer", "silu", True, True, "rms", F32, seed=T), "layer", "silu", "rms")


def test_a_mean_far_above_the_spread():
    """Rows around 300 with a spread of 1: the variance is taken about the mean, so fp32
    keeps it (a difference of squares would lose 17 bits): 2^-24 * 300 of each deviation."""
    i = _inputs(2, 9, 768, 1, "layer", "none", False, False, "none", F32, mean=300.0)
    h, _, _ = _run(i, "layer", "none", "none")
    hr, _, _ = _formula(i, "layer", "none", "none", 1.0)
    assert _rel(h, hr) <= 300 * 2.0 ** -22
    i = _inputs(2, 9, 64, 1, "layer", "none", False, False, "none", F32, mean=300.0)
    h, _, _ = _run(i, "layer", "none", "none")
    hr, _, _ = _formula(i, "layer", "none", "none", 1.0)
    assert _rel(h, hr) <= 300 * 2.0 ** -22


def test_constant_and_extreme_rows():
    """A row of zeros and a constant row stay finite (eps), the gate at the type's lowest and
    highest values saturates, and a NaN or infinite row touches no other row."""
    i = _inputs(1, 8, 768, 1, "layer", "silu", True, True, "rms", BF)
    i["y"][0, 1] = 0
    i["y"][0, 2] = 5
    i["x"][0, 1] = 0
    i["gate"][0, 3] = torch.finfo(BF).min
    i["gate"][0, 4] = 100.0
    clean = _run(i, "layer", "silu", "rms")
    assert all(bool(t.isfinite().all()) for t in (clean[0], clean[1], *(t for t in clean[2] if t is not None)))
    assert torch.equal(clean[0][0, 3], i["x"][0, 3])  # SiLU of the lowest value: -0 * p
    i["y"][0, 6] = float("nan")
    i["x"][0, 7] = float("inf")
    h, u, g = _run(i, "layer", "silu", "rms")
    for a, b in ((h, clean[0]), (u, clean[1]), (g.y, clean[2].y), (g.x, clean[2].x), (g.gate, clean[2].gate)):
        assert torch.equal(a[0, :6], b[0, :6])
    assert bool(h[0, 6].isnan().all())


@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu"])
def test_gate_at_its_extremes(act):
    gate = torch.tensor([-3.0e38, -90.0, -20.0, -6.0, -1e-30, 0.0, 1e-30, 6.0, 20.0, 90.0, 3.0e38, -12.0], device="cuda")
    y = torch.full((1, 1, 12), 1.0, device="cuda")
    h, _, st = abi.ttt_block_norm_fwd(y, gate=gate.view(1, 1, -1), act=act, want_stats=True)
    g = abi.ttt_block_norm_bwd(y, None, y, st, gate=gate.view(1, 1, -1), act=act)
    abi.ttt_sync_status()
    gd = gate.double().cpu().requires_grad_(True)
    f = {"sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[act](gd)
    f.sum().backward()
    for got, ref in ((h.view(-1), f.detach()), (g.gate.view(-1), gd.grad)):
        ok = ref.abs() < 1e37
        assert bool(got.cpu()[ok].isfinite().all())
        assert float((got.double().cpu() - ref)[ok].abs().max()) <= 2.0 ** -20 * max(1.0, float(ref[ok].abs().max()))


def test_gradients_against_differences():
    """Directional differences of the kernel's forward in fp32, step 2^-6: error
    O(step^2) = 2.4e-4 of third derivatives of order one, plus rounding 2^-22 / step."""
    for post, act, pre in (("layer", "gelu", "rms"), ("rms", "silu", "layer")):
        i = _inputs(2, 5, 96, 3, post, act, True, True, pre, F32, seed=3)
        _, _, g = _run(i, post, act, pre)

        def objective(j):
            h, u, _ = _run(j, post, act, pre)
            return float((h.double() * i["dh"].double()).sum() + (u.double() * i["du"].double()).sum())
        gen = torch.Generator().manual_seed(5)
        for n in ("y", "x", "gate") + VEC:
            if i[n] is None:
                continue
            v = torch.randn(i[n].shape, generator=gen).cuda()
            v = v / v.norm()
            e = 2.0 ** -6
            j = dict(i)
            j[n] = i[n] + e * v
            hi = objective(j)
            j[n] = i[n] - e * v
            lo = objective(j)
            want = float((getattr(g, n).double() * v.double()).sum())
            scale = float(getattr(g, n).double().norm())
            assert abs((hi - lo) / (2 * e) - want) <= 4e-3 * max(1.0, scale), n


def test_strided_and_broadcast_inputs_and_h_over_x():
    B, T, D = 3, 17, 128
    i = _inputs(B, T, D, 1, "rms", "silu", True, True, "rms", BF, seed=8)
    wide = torch.randn(B, T, 3 * D + 8, device="cuda").to(BF)
    j = dict(i, gate=wide[..., D:2 * D], x=wide[:, :1, :D].expand(B, T, D))
    _check(j, "rms", "silu", "rms")
    odd = torch.randn(B, T, D + 1, device="cuda").to(BF)[..., :D]  # rows 258 bytes apart
    _check(dict(i, y=odd), "rms", "silu", "rms")
    kw = dict(gate=i["gate"], act="silu", post="rms", pre="rms", **{n: i[n] for n in VEC})
    want = abi.ttt_block_norm_fwd(i["y"], x=i["x"], **kw)
    x = i["x"].clone()
    got = abi.ttt_block_norm_fwd(i["y"], x=x, h=x, **kw)
    abi.ttt_sync_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0].data_ptr() == x.data_ptr()


def test_same_bits_every_run_and_no_dh():
    i = _inputs(4, 700, 768, 12, "layer", "gelu", True, True, "layer", BF, seed=4)
    a, b = _run(i, "layer", "gelu", "layer"), _run(i, "layer", "gelu", "layer")
    assert all(torch.equal(s, t) for s, t in zip((a[0], a[1], *a[2]), (b[0], b[1], *b[2])))
    _check(dict(i, dh=None), "layer", "gelu", "layer")


def test_no_tokens():
    w = torch.ones(64, device="cuda")
    y = torch.empty(0, 5, 64, device="cuda", dtype=BF)
    h, u, st = abi.ttt_block_norm_fwd(y, post="rms", post_weight=w, want_stats=True)
    g = abi.ttt_block_norm_bwd(h, None, y, st, post="rms", post_weight=w)
    abi.ttt_sync_status()
    assert h.shape == y.shape and u is None and bool((g.post_weight == 0).all())


def test_full_size_every_token():
    """The 125M layer's batch, forward and backward, all 16384 tokens."""
    _check(_inputs(8, 2048, 768, 12, "layer", "gelu", True, True, "rms", BF, seed=6), "layer", "gelu", "rms")


def test_on_a_side_stream():
    i = _inputs(2, 300, 768, 12, "layer", "silu", True, True, "rms", BF)
    want = _run(i, "layer", "silu", "rms")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kw = dict(x=i["x"], gate=i["gate"], act="silu", post="layer", pre="rms", **{n: i[n] for n in VEC})
    with torch.cuda.stream(st):
        h, u, s = abi.ttt_block_norm_fwd(i["y"], want_stats=True, **kw)
        g = abi.ttt_block_norm_bwd(i["dh"], i["du"], i["y"], s, **kw)
    abi.ttt_sync_status(st)
    for a, b in zip((h, u, *g), (want[0], want[1], *want[2])):
        assert (a is None and b is None) or torch.equal(a, b)
