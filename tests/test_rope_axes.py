"""Positions with several axes without a GPU: the pairs' axes, the table, and the refusals of
ttt_rope_axes at the C boundary and in the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

from test_sequence_layers_gb300 import abi, build, rotary
from tests.test_rotary import FAKE, _Dev


@pytest.fixture(scope="module")
def L():
    build.build()
    return abi.lib()


def test_the_axes_of_the_pairs():
    assert list(rotary.rope_axes((2, 1, 1))) == [0, 0, 1, 2]
    assert list(rotary.rope_axes((3, 1, 2), "cyclic")) == [0, 1, 2, 0, 2, 0]
    assert rotary.rope_axes((0, 2)) == bytes((1, 1))
    for bad in ((), (2, -1)):
        with pytest.raises(ValueError):
            rotary.rope_axes(bad)
    with pytest.raises(ValueError):
        rotary.rope_axes((2, 2), "diagonal")


def test_table():
    axis = rotary.rope_axes((3, 2), "cyclic")  # 0 1 0 1 0
    t = rotary.rope_axes_table(20, axis, device="cpu").double()
    seen = [0, 0]
    for i, a in enumerate(axis):
        ang = 13 * 10000.0 ** (-seen[a] / (3, 2)[a])
        seen[a] += 1
        assert abs(float(t[13, i, 0]) - math.cos(ang)) <= 2.0 ** -24 and abs(float(t[13, i, 1]) - math.sin(ang)) <= 2.0 ** -24
    assert torch.equal(rotary.rope_axes_table(20, axis, per_axis=False, device="cpu"), rotary.rope_table(20, 10, device="cpu"))
    lin = rotary.rope_axes_table(20, axis, device="cpu", scaling="linear", factor=2.0)
    assert torch.allclose(lin[::2], rotary.rope_axes_table(10, axis, device="cpu"), atol=2.0 ** -22)


def _call(L, axes=3, grid=(4, 5, 6, 1), stride=0, pair_axis=bytes(32), q=FAKE, pos=None, qo=FAKE + (1 << 30), **kw):
    d = dict(B=2, T=4, Hq=3, Hk=3, d=64, rot=64, interleaved=0, inverse=0, io_dtype=abi.TTT_BF16, table_rows=8,
             period=0, pos0=0, positions_batch_stride=0)
    d.update(kw)
    std = [d["Hq"] * d["T"] * d["d"], d["T"] * d["d"], d["d"]]
    desc = abi.RopeAxesDesc(*d.values(), (ctypes.c_longlong * 18)(*(std * 6)), axes, (ctypes.c_int * 4)(*grid), stride)
    return L.ttt_rope_axes(desc, pair_axis, q, None, None, FAKE + (1 << 31), pos, qo, None, None, None)


def test_refusals(L):
    assert L.ttt_rope_axes(*[None] * 11) == -1
    for bad in (dict(axes=0), dict(axes=5), dict(pair_axis=None), dict(pair_axis=bytes(31) + b"\3"), dict(period=4),
                dict(grid=(4, 5, 0, 1)), dict(grid=(4, 9, 6, 1)), dict(pos0=117), dict(pos0=-1), dict(T=121),
                dict(pos=FAKE + (1 << 32), stride=-1), dict(q=None), dict(rot=66), dict(B=-1),
                dict(pos=FAKE + (1 << 30), stride=4)):
        assert _call(L, **bad) == -1, bad
    assert _call(L, grid=(7, 7, 7, 7), axes=4, table_rows=7, pair_axis=bytes(32), B=0) == 0
    assert _call(L, d=1026, rot=2) == -2
    assert _call(L, pos=FAKE + (1 << 32) + 4, stride=8) == -3


@pytest.mark.parametrize("bad", [
    dict(grid=None), dict(positions=_Dev((2, 2, 4), torch.int64)), dict(grid=(1,) * 5), dict(grid=()),
    dict(pair_axis=bytes(7)), dict(grid=None, positions=_Dev((2, 3, 4), torch.int64)),
    dict(grid=None, positions=_Dev((2, 2, 4), torch.int32)), dict(grid=None, positions=_Dev((4,), torch.int64)),
    dict(grid=None, positions=_Dev((5, 2, 4), torch.int64)), dict(table=_Dev((9, 8), torch.float32)),
    dict(q=_Dev((2, 3, 4, 16), torch.float16)),
])
def test_binding_refuses_before_any_launch(bad):
    a = dict(q=_Dev((2, 3, 4, 16)), k=_Dev((2, 3, 4, 16)), v=None, table=_Dev((9, 8, 2), torch.float32), pair_axis=bytes(8),
             grid=(2, 2), q_out=_Dev((2, 3, 4, 16)), k_out=_Dev((2, 3, 4, 16)))
    a.update(bad)
    with pytest.raises(ValueError):
        abi.ttt_rope_axes(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("table"), a.pop("pair_axis"), **a)


@pytest.mark.parametrize("bad", [8, "01010101", [0.5] * 8, [-1] * 8, [256] * 8, torch.zeros(8)])
def test_pair_axes_that_are_no_sequence_of_axes(bad):
    """A number above all: bytes(8) is eight zeros, a rotation by the first axis alone."""
    a = dict(k=None, v=None, table=_Dev((9, 8, 2), torch.float32), grid=(2, 2), q_out=_Dev((2, 3, 4, 16)))
    with pytest.raises(ValueError):
        abi.ttt_rope_axes(_Dev((2, 3, 4, 16)), pair_axis=bad, **a)
    with pytest.raises(ValueError):
        rotary.rope_axes_table(9, bad, device="cpu")


@pytest.mark.parametrize("seq", [[0, 1, 1, 0], (0, 1, 1, 0), np.array([0, 1, 1, 0]), torch.tensor([0, 1, 1, 0]), range(4)])
def test_sequences_of_axes(seq, monkeypatch):
    got = []
    monkeypatch.setattr(_Dev, "data_ptr", lambda self: FAKE)
    monkeypatch.setattr(abi, "_call", lambda name, di, desc, axis, *rest: got.append(axis))
    q = _Dev((2, 3, 4, 8))
    abi.ttt_rope_axes(q, None, None, _Dev((9, 4, 2), torch.float32), seq, grid=(2, 2, 1, 1), q_out=_Dev((2, 3, 4, 8)))
    want = bytes(int(a) for a in seq)
    assert got == [want]
    assert torch.equal(rotary.rope_axes_table(9, seq, device="cpu"), rotary.rope_axes_table(9, want, device="cpu"))
