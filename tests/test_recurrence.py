"""Refusals of the gated linear recurrence at the C boundary and in the binding, without
a GPU."""
import ctypes

import pytest
import torch

from test_sequence_layers_gb300 import abi, build
from tests.test_rotary import _Dev

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    build.build()
    return abi.lib()


def _at(i):
    return (1 << 20) + i * (1 << 24)


def _desc(**kw):
    d = dict(B=2, T=300, C=64, io_dtype=abi.TTT_BF16, mode=2)
    d.update(kw)
    return abi.RecurrenceDesc(*d.values(), (ctypes.c_longlong * 6)(*([d["T"] * d["C"], d["C"]] * 3)))


def _fwd(L, x=_at(1), f=_at(2), reset=None, h0=None, h=_at(3), h_last=None, states=None, **kw):
    return L.ttt_recurrence_fwd(_desc(**kw), x, f, reset, h0, h, h_last, states, None)


def _bwd(L, dh=_at(1), x=_at(2), f=_at(3), reset=None, states=_at(4), dh_last=None, dx=_at(5), df=_at(6), dh0=None, **kw):
    return L.ttt_recurrence_bwd(_desc(**kw), dh, x, f, reset, states, dh_last, dx, df, dh0, None)


def test_forward_refusals(L):
    assert L.ttt_recurrence_fwd(None, None, None, None, None, None, None, None, None) == -1
    for bad in (dict(B=-1), dict(T=-1), dict(C=0), dict(mode=3), dict(mode=-1), dict(io_dtype=2), dict(x=None),
                dict(f=None), dict(h=None), dict(h=_at(1)), dict(h=_at(2) + 32), dict(h_last=_at(1)),
                dict(h0=_at(4), h_last=_at(4) + 16), dict(states=_at(3)), dict(states=_at(4), h0=_at(4)),
                dict(reset=_at(3))):
        assert _fwd(L, **bad) == -1, bad
    assert _fwd(L, B=70000) == -2
    assert _fwd(L, B=0) == 0 and _fwd(L, T=0) == 0
    for bad in (dict(x=_at(1) + 1), dict(h=_at(3) + 1), dict(h0=_at(4) + 2), dict(states=_at(4) + 1)):
        assert _fwd(L, **bad) == -3, bad


def test_backward_refusals(L):
    for bad in (dict(dx=None), dict(df=None), dict(states=None), dict(dx=_at(6)), dict(dx=_at(1)), dict(df=_at(4)),
                dict(dh0=_at(5)), dict(dh0=_at(7), dh_last=_at(7)), dict(x=None), dict(T=-1)):
        assert _bwd(L, **bad) == -1, bad
    for bad in (dict(dh=_at(1) + 1), dict(dx=_at(5) + 1), dict(dh_last=_at(7) + 2)):
        assert _bwd(L, **bad) == -3, bad
    assert _bwd(L, B=0) == 0


@pytest.mark.parametrize("bad", [
    dict(x=_Dev((2, 9))), dict(x=_Dev((2, 9, 8), cuda=False)), dict(x=_Dev((2, 9, 8), torch.float16)),
    dict(f=_Dev((2, 9, 8), F32)), dict(f=_Dev((2, 8, 8))), dict(f=_Dev((2, 9, 8), last=3)), dict(h0=_Dev((2, 8), BF)),
    dict(h0=_Dev((8,), F32)), dict(reset=_Dev((2, 9), F32)), dict(reset=_Dev((9,), torch.bool)), dict(h=_Dev((2, 9, 9))),
    dict(h_last=_Dev((2, 9), F32)), dict(states=_Dev((2, 2, 8), F32)), dict(x=_Dev((2, 9, 8), index=1)),
])
def test_binding_refuses_before_any_launch(bad):
    a = dict(x=_Dev((2, 9, 8)), f=_Dev((2, 9, 8)), h=_Dev((2, 9, 8)), h_last=_Dev((2, 8), F32),
             states=_Dev((2, 1, 8), F32))
    a.update(bad)
    with pytest.raises(ValueError):
        abi.ttt_recurrence_fwd(a.pop("x"), a.pop("f"), **a)
