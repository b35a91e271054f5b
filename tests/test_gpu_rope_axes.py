"""Rotary positions with several axes on the GPU against the rotation in 64 bits.  A result is
two products and a sum of entries below their size, in fp32: 3 * 2^-24 of |a| + |b|, times the
table's factor, and one rounding to its type."""
import pytest
import torch

from test_sequence_layers_gb300 import abi, rotary
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _ref(x, table, axis, pos, interleaved, inverse):
    """(value, slack); pos: [axes,B,T]."""
    x = x.double()
    half = len(axis)
    where = pos[list(axis)].permute(1, 2, 0)
    cs = table.double()[where, torch.arange(half, device="cuda")][:, None]
    c, s = cs[..., 0], cs[..., 1] * (-1 if inverse else 1)
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (rot[..., 0::2], rot[..., 1::2]) if interleaved else (rot[..., :half], rot[..., half:])
    y, m = (a * c - b * s, a * s + b * c), a.abs() + b.abs()
    join = (lambda u, v: torch.stack([u, v], -1).flatten(-2)) if interleaved else (lambda u, v: torch.cat([u, v], -1))
    return torch.cat([join(*y), rest], -1), torch.cat([join(m, m), 0 * rest], -1) * 3 * 2.0 ** -24


def _close(got, ref, slack):
    u = torch.finfo(got.dtype).eps / 2
    assert bool(((got.double() - ref).abs() <= u * ref.abs() * (1 + 2.0 ** -6) + slack).all())


def _grid(extents, B, pos0, T):
    t = torch.arange(pos0, pos0 + T, device="cuda")
    out = []
    for n in reversed(extents):
        out.insert(0, t % n)
        t = t // n
    return torch.stack(out)[:, None].expand(-1, B, -1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["blocks", "cyclic"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,Hk,d,sections,grid,pos0,T", [
    (3, 3, 64, (16, 16), (14, 14), 0, 196), (4, 1, 64, (16, 8, 8), (3, 5, 4), 7, 50), (2, 2, 128, (16, 24, 24), (2, 9, 1), 0, 18),
    (1, 1, 20, (3, 2), (6, 6), 30, 6), (2, 3, 48, (8, 0, 8), (1, 1, 30), 0, 30), (1, 2, 34, (1, 1, 1, 1), (2, 2, 2, 2), 3, 13),
    (5, 5, 16, (8,), (40,), 0, 40)])
def test_grids(H, Hk, d, sections, grid, pos0, T, interleaved, layout, dtype):
    B = 2
    axis = rotary.rope_axes(sections, layout)
    table = rotary.rope_axes_table(max(grid) + 3, axis)
    q, k, v = (torch.randn(B, h, T, d, device="cuda").to(dtype) for h in (H, Hk, Hk))
    pos = _grid(grid, B, pos0, T)
    for inverse in (False, True):
        out = abi.ttt_rope_axes(q, k, v, table, axis, grid=grid, pos0=pos0, interleaved=interleaved, inverse=inverse)
        for got, x in zip(out, (q, k)):
            _close(got, *_ref(x, table, axis, pos, interleaved, inverse))
        assert torch.equal(out[2], v)
        # given positions: the same bits, per sequence or shared by the batch
        for p in (pos.contiguous(), pos[:, 0].contiguous()):
            again = abi.ttt_rope_axes(q, k, v, table, axis, positions=p, interleaved=interleaved, inverse=inverse)
            assert all(torch.equal(a, b) for a, b in zip(out, again))
    abi.ttt_sync_status()


def test_one_axis_is_ttt_rope():
    table = rotary.rope_table(100, 32)
    q, k, v = (torch.randn(2, 3, 50, 64, device="cuda").to(BF) for _ in range(3))
    want = abi.ttt_rope(q, k, v, table, pos0=9)
    got = abi.ttt_rope_axes(q, k, v, rotary.rope_axes_table(100, bytes(16)), bytes(16), grid=(100,), pos0=9)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # equal positions on every axis: one axis' frequencies, text between pictures
    axis = rotary.rope_axes((6, 5, 5), "cyclic")
    pos = torch.randint(0, 100, (2, 50), device="cuda")
    want = abi.ttt_rope(q, k, v, table, positions=pos)
    got = abi.ttt_rope_axes(q, k, v, rotary.rope_axes_table(100, axis, per_axis=False), axis, positions=pos.expand(3, -1, -1).contiguous())
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_inverse_undoes_and_layouts():
    """Token-major projections in, head-major out, the gradients back into one token-major buffer."""
    B, T, H, d = 2, 60, 3, 32
    axis = rotary.rope_axes((4, 6, 6))
    table = rotary.rope_axes_table(32, axis)
    qkv = torch.randn(B, T, 3, H, d, device="cuda")
    out = abi.ttt_rope_axes(*qkv.permute(2, 0, 3, 1, 4).unbind(0), table, axis, grid=(4, 5, 3))
    back = torch.empty_like(qkv)
    q, k, v = back.permute(2, 0, 3, 1, 4).unbind(0)
    abi.ttt_rope_axes(*out, table, axis, grid=(4, 5, 3), inverse=True, q_out=q, k_out=k, v_out=v)
    # twice the rotation's error, and c^2 + s^2 within 2^-23 of one
    assert bool(((back - qkv).abs() <= 2.0 ** -20 * qkv.abs().max()).all())
    # in place
    q2, k2 = out[0].clone(), out[1].clone()
    abi.ttt_rope_axes(q2, k2, None, table, axis, grid=(4, 5, 3), inverse=True, q_out=q2, k_out=k2)
    assert torch.equal(q2, q) and torch.equal(k2, k)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_position_out_of_range_touches_its_axis_alone(dtype):
    axis = rotary.rope_axes((8, 8))
    table = rotary.rope_axes_table(10, axis)
    q = torch.randn(1, 2, 4, 32, device="cuda").to(dtype)
    pos = torch.tensor([[0, 9, 10, -1], [3, 1 << 40, 5, 9]], device="cuda")
    got = abi.ttt_rope_axes(q, None, None, table, axis, positions=pos)[0]
    with pytest.raises(abi.TTTError) as e:
        abi.ttt_sync_status()
    assert e.value.code == -7
    ok = abi.ttt_rope_axes(q, None, None, table, axis, positions=pos.clamp(0, 9))[0]
    abi.ttt_sync_status()
    bad = torch.zeros(4, 32, dtype=torch.bool, device="cuda")
    bad[2:, 0:8] = bad[2:, 16:24] = True    # axis 0 of tokens 2 and 3
    bad[1, 8:16] = bad[1, 24:32] = True     # axis 1 of token 1
    assert bool(torch.isnan(got[..., bad]).all()) and torch.equal(got[..., ~bad], ok[..., ~bad])


def test_decoding_and_many_heads():
    axis = rotary.rope_axes((16, 8, 8), "cyclic")
    table = rotary.rope_axes_table(2000, axis)
    for B, H, T in ((64, 12, 1), (1, 700, 1), (1, 2, 3)):
        q, k = (torch.randn(B, H, T, 64, device="cuda").to(BF) for _ in range(2))
        pos = torch.randint(0, 2000, (3, B, T), device="cuda")
        out = abi.ttt_rope_axes(q, k, None, table, axis, positions=pos)
        for got, x in zip(out, (q, k)):
            _close(got, *_ref(x, table, axis, pos, False, False))
    assert out[2] is None
