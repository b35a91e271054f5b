"""Rotary positions on the GPU against the rotation in 64 bits.

Tolerance, from the arithmetic: an output is one rounding to the I/O type (2^-9 of its
value in bf16, 2^-24 in fp32) of two fp32 products and a sum (2 ulp of |a| + |b|, with
|cos|, |sin| <= 1.14 with YaRN's factor): |err| <= u |y| + 2^-22 (|a| + |b|), u = 2^-8 or
0 (the fp32 rounding is inside the second term)."""
import numpy as np
import pytest
import torch

from test_sequence_layers_gb300 import abi, rotary
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _ref(x, table, pos, interleaved, inverse):
    """Rotation in 64 bits of [B,H,T,d]; also |a| + |b| of every output."""
    x = x.double().cpu()
    rot = 2 * table.shape[1]
    tab = table.double().cpu()[pos]               # [B,T,rot/2,2]
    y, mag = x.clone(), torch.zeros_like(x)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = tab[:, None, :, i, 0], tab[:, None, :, i, 1] * (-1 if inverse else 1)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def _close(got, ref, mag):
    u = 2.0 ** -8 if got.dtype == BF else 0.0
    err = (got.double().cpu() - ref).abs()
    assert bool((err <= u * ref.abs() + 2.0 ** -22 * mag).all()), float((err - u * ref.abs()).max())


def _check(B, T, Hq, Hk, d, rot, dtype, interleaved, inverse, fused=True, given=False, period=0, seed=0, scaling="none"):
    g = torch.Generator().manual_seed(seed)
    rows = period if period else T + 37
    table = rotary.rope_table(rows, rot, scaling=scaling, factor=4.0 if scaling != "none" else 1.0)
    if fused:
        buf = torch.randn(B, T, Hq + 2 * Hk, d, generator=g).to(dtype).cuda()
        q, k, v = (t.transpose(1, 2) for t in buf.split([Hq, Hk, Hk], 2))
    else:
        q, k, v = (torch.randn(B, h, T, d, generator=g).to(dtype).cuda() for h in (Hq, Hk, Hk))
    pos, kw = torch.arange(T)[None].repeat(B, 1), {}
    if given:
        pos = torch.randint(0, 4 * rows if period else rows, (B, T), generator=g)
        kw["positions"] = pos.cuda()
    else:
        pos = pos + 11
        kw["pos0"] = 11
    kept = [t.clone() for t in (q, k, v)]
    out = abi.ttt_rope(q, k, v, table, interleaved=interleaved, inverse=inverse, period=period, **kw)
    abi.ttt_sync_status()
    if period:
        pos = pos % period
    for got, t in zip(out[:2], (q, k)):
        assert got.is_contiguous() and got.shape == t.shape
        _close(got, *_ref(t, table, pos, interleaved, inverse))
    assert torch.equal(out[2], v)
    assert all(torch.equal(a, b) for a, b in zip(kept, (q, k, v)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 32), (128, 128), (16, 16), (20, 20), (20, 10), (12, 4), (7, 6), (5, 2),
                                   (64, 0), (96, 40), (1, 0), (1024, 512)])
def test_head_sizes_and_layouts(d, rot, interleaved, dtype):
    _check(2, 33, 3, 3, d, rot, dtype, interleaved, False, seed=d + rot)
    _check(1, 5, 4, 2, d, rot, dtype, interleaved, True, fused=False, given=True, seed=d * rot)


@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (64, 1, 12, 12), (1, 1000, 1, 1), (3, 257, 7, 1), (2, 2048, 12, 12),
                                       (1, 16, 32, 4)])
def test_batches_and_lengths(B, T, Hq, Hk):
    for period, scaling in ((0, "yarn"), (16, "none")):
        _check(B, T, Hq, Hk, 64, 64, BF, False, False, given=B > 2, period=period, scaling=scaling, seed=T)


def test_inverse_undoes_the_rotation_into_the_projection_buffer():
    """Forward from a [B,T,3,H,d] buffer and back into another: fp32 to a few ulp, and the
    gradient pairing <rope(x), g> = <x, rope^-1(g)> that makes it the backward pass."""
    B, T, H, d = 2, 50, 5, 64
    table = rotary.rope_table(T, 48)
    qkv = torch.randn(B, T, 3, H, d, device="cuda")
    q, k, v = qkv.permute(2, 0, 3, 1, 4).unbind(0)
    out = abi.ttt_rope(q, k, v, table)
    back = torch.empty_like(qkv)
    bq, bk, bv = back.permute(2, 0, 3, 1, 4).unbind(0)
    abi.ttt_rope(*out, table, inverse=True, q_out=bq, k_out=bk, v_out=bv)
    abi.ttt_sync_status()
    assert float((back - qkv).abs().max()) <= 2.0 ** -19
    gq = torch.randn_like(out[0])
    dq = abi.ttt_rope(gq, None, None, table, inverse=True)[0]
    a, b = (out[0].double() * gq.double()).sum(), (q.double() * dq.double()).sum()
    assert abs(float(a - b)) <= 1e-5 * float((out[0].double() * gq.double()).abs().sum())


def test_in_place_and_single_tensors():
    B, T, H, d = 2, 19, 3, 32
    table = rotary.rope_table(64, 32)
    x = torch.randn(B, T, 2, H, d, device="cuda").to(BF)
    q, k = x.permute(2, 0, 3, 1, 4).unbind(0)
    want = abi.ttt_rope(q, k, None, table, pos0=40)
    got = abi.ttt_rope(q, k, None, table, pos0=40, q_out=q, k_out=k)
    abi.ttt_sync_status()
    assert got[2] is None and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    only = abi.ttt_rope(want[0], None, None, table)
    assert only[1] is None and only[0].shape == want[0].shape


def test_broadcast_input_and_odd_strides():
    table = rotary.rope_table(9, 16)
    base = torch.randn(9, 17, device="cuda").to(BF)[:, :16]  # rows 34 bytes apart
    q = base[None, None].expand(2, 3, 9, 16)
    out = abi.ttt_rope(q, None, None, table)[0]
    abi.ttt_sync_status()
    _close(out, *_ref(q, table, torch.arange(9)[None].repeat(2, 1), False, False))


def test_a_position_outside_the_table_is_reported():
    B, T, H, d = 2, 6, 2, 64
    table = rotary.rope_table(32, 32)
    q = torch.randn(B, H, T, d, device="cuda").to(BF)
    pos = torch.arange(T, device="cuda").repeat(B, 1)
    for bad in (32, -1, 1 << 40):
        p = pos.clone()
        p[1, 3] = bad
        out = abi.ttt_rope(q, None, None, table, positions=p)[0]
        with pytest.raises(abi.TTTError) as e:
            abi.ttt_sync_status()
        assert e.value.code == -7
        assert bool(out[1, :, 3, :32].isnan().all()) and torch.equal(out[1, :, 3, 32:], q[1, :, 3, 32:])
        out[1, :, 3] = 0
        assert not bool(out.isnan().any())
    abi.ttt_sync_status()  # reported once
    ok = pos + (1 << 40)
    a = abi.ttt_rope(q, None, None, table, positions=ok, period=32)[0]
    b = abi.ttt_rope(q, None, None, table, period=32)[0]
    abi.ttt_sync_status()
    assert torch.equal(a, b)


def test_empty_and_refused():
    table = rotary.rope_table(8, 16)
    q = torch.empty(0, 2, 4, 16, device="cuda", dtype=BF)
    assert abi.ttt_rope(q, None, None, table)[0].shape == q.shape
    q = torch.zeros(1, 2, 9, 16, device="cuda", dtype=BF)
    with pytest.raises(abi.TTTError) as e:
        abi.ttt_rope(q, None, None, table)
    assert e.value.code == -1


def test_on_a_side_stream():
    table = rotary.rope_table(300, 64)
    q = torch.randn(2, 12, 300, 64, device="cuda").to(BF)
    want = abi.ttt_rope(q, None, None, table)[0]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = abi.ttt_rope(q, None, None, table, stream=st)[0]
    abi.ttt_sync_status(st)
    assert torch.equal(got, want)
