"""Rotary positions without a GPU: the table against its definition, and the refusals of
ttt_rope at the C boundary and in the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

from test_sequence_layers_gb300 import abi, build, rotary

FAKE = 1 << 20


@pytest.fixture(scope="module")
def L():
    build.build()
    return abi.lib()


def test_table_is_the_definition_rounded_once():
    t = rotary.rope_table(50, 12, device="cpu").double().numpy()
    for p in (0, 1, 49):
        for i in range(6):
            a = p * 10000.0 ** (-2.0 * i / 12)
            assert abs(t[p, i, 0] - math.cos(a)) <= 2.0 ** -24 and abs(t[p, i, 1] - math.sin(a)) <= 2.0 ** -24
    assert rotary.rope_table(7, 0, device="cpu").shape == (7, 0, 2)


def test_long_positions_keep_their_angle():
    """Position 10^6 of the fastest pair: cos(10^6), which an fp32 product of position and
    frequency also has, and of the second pair, which it has not."""
    inv, _ = rotary.rope_frequencies(64)
    pos = 1000003
    ang = pos * inv
    t = (torch.stack([ang.cos(), ang.sin()], -1)).float()
    assert abs(float(t[0, 0]) - math.cos(pos)) < 1e-7
    assert abs(float(t[1, 1]) - math.sin(pos * 10000.0 ** (-2.0 / 64))) < 1e-7


def test_scalings():
    base, one = rotary.rope_frequencies(64)
    assert one == 1.0
    lin, m = rotary.rope_frequencies(64, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin, base / 4, rtol=1e-15)
    ntk, m = rotary.rope_frequencies(64, scaling="ntk", factor=4.0)
    assert m == 1.0 and abs(ntk[0] / base[0] - 1) < 1e-12 and abs(ntk[-1] * 4 / base[-1] - 1) < 1e-12
    yarn, m = rotary.rope_frequencies(64, scaling="yarn", factor=4.0, original_rows=4096)
    assert abs(m - (0.1 * math.log(4) + 1)) < 1e-12
    turns = 4096 * base / (2 * math.pi)
    for i in range(32):
        if turns[i] >= 32:
            assert yarn[i] == base[i]
        elif turns[i] <= 1:
            assert abs(yarn[i] - base[i] / 4) < 1e-15
        else:
            assert base[i] / 4 < yarn[i] < base[i]
    for bad in (dict(rot=5), dict(rot=8, scaling="cubic"), dict(rot=8, factor=0.0),
                dict(rot=8, scaling="yarn", factor=2.0, beta_fast=1.0)):
        with pytest.raises(ValueError):
            rotary.rope_frequencies(**bad)


def _call(L, q=FAKE, k=None, v=None, table=FAKE, pos=None, qo=FAKE + (1 << 30), ko=None, vo=None, strides=None, **kw):
    d = dict(B=2, T=4, Hq=3, Hk=3, d=64, rot=64, interleaved=0, inverse=0, io_dtype=abi.TTT_BF16, table_rows=8,
             period=0, pos0=0, positions_batch_stride=0)
    d.update(kw)
    std = [d["Hq"] * d["T"] * d["d"], d["T"] * d["d"], d["d"]]
    desc = abi.RopeDesc(*d.values(), (ctypes.c_longlong * 18)(*(strides or std * 6)))
    return L.ttt_rope(desc, q, k, v, table, pos, qo, ko, vo, None)


def test_refusals(L):
    assert L.ttt_rope(None, None, None, None, None, None, None, None, None, None) == -1
    for bad in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(d=0), dict(rot=3), dict(rot=66), dict(interleaved=2),
                dict(inverse=-1), dict(io_dtype=3), dict(period=9), dict(pos0=-1), dict(pos0=5), dict(q=None),
                dict(qo=None), dict(table=None), dict(k=FAKE), dict(k=FAKE, ko=FAKE + (1 << 28), Hk=0),
                dict(table_rows=3)):
        assert _call(L, **bad) == -1, bad
    assert _call(L, d=1026, rot=2) == -2
    assert _call(L, B=0) == 0 and _call(L, T=0) == 0
    assert _call(L, q=FAKE + 1) == -3
    assert _call(L, qo=FAKE + (1 << 30) + 1) == -3
    assert _call(L, table=FAKE + 4) == -3
    assert _call(L, qo=FAKE + 64) == -1                                   # a shifted output over its input
    std = [768, 256, 64]
    assert _call(L, strides=std * 3 + [0, 256, 64] + std * 2) == -1       # an output written twice
    assert _call(L, strides=[-768, 256, 64] + std * 5) == -1


class _Dev:
    def __init__(self, shape, dtype=torch.bfloat16, cuda=True, index=0, last=1):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, cuda
        self.device = torch.device("cuda", index) if cuda else torch.device("cpu")
        self.last = last

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def stride(self, i=None):
        s = [self.last]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def is_contiguous(self):
        return self.last == 1

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        raise AssertionError("the binding reached the library with a bad argument")


@pytest.mark.parametrize("bad", [
    dict(q=_Dev((2, 3, 4, 16), cuda=False)), dict(q=_Dev((2, 3, 4))), dict(q=_Dev((2, 3, 4, 16), torch.float16)),
    dict(q=_Dev((2, 3, 4, 16), last=2)), dict(k=_Dev((2, 3, 5, 16))), dict(k=_Dev((2, 3, 4, 16), torch.float32)),
    dict(v=_Dev((2, 2, 4, 16))), dict(v=_Dev((2, 3, 4, 16), index=1)), dict(table=_Dev((9, 8), torch.float32)),
    dict(table=_Dev((9, 8, 2))), dict(positions=_Dev((2, 4), torch.int32)), dict(positions=_Dev((3, 4), torch.int64)),
    dict(q_out=_Dev((2, 3, 4, 8))), dict(k=None, v=None, k_out=_Dev((2, 3, 4, 16))),
])
def test_binding_refuses_before_any_launch(bad):
    a = dict(q=_Dev((2, 3, 4, 16)), k=_Dev((2, 3, 4, 16)), v=_Dev((2, 3, 4, 16)),
             table=_Dev((9, 8, 2), torch.float32), q_out=_Dev((2, 3, 4, 16)), k_out=_Dev((2, 3, 4, 16)),
             v_out=_Dev((2, 3, 4, 16)))
    if "k_out" in bad:
        a["v_out"] = None
    a.update(bad)
    with pytest.raises(ValueError):
        abi.ttt_rope(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("table"), **a)
