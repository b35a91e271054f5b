"""Refusals of the short convolution and the selective scan at the C boundary and in the
binding, their packed descriptors, and whose memory a call on another stream takes, without a
GPU."""
import ctypes

import pytest
import torch

from test_sequence_layers_gb300 import abi, build, rotary
from tests.test_descriptors import test_same_bytes as same_bytes
from tests.test_rotary import _Dev
from tests.test_streams import _T, _check, gpu  # noqa: F401

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    build.build()
    return abi.lib()


def _at(i):
    return (1 << 20) + i * (1 << 24)


@pytest.mark.parametrize("packed,struct", [(abi._AXES_DESC, abi.RopeAxesDesc), (abi._CONV_DESC, abi.ShortConvDesc),
                                           (abi._SCAN_DESC, abi.ScanDesc), (abi._THREE, abi.ScanVectors)])
def test_packed_descriptors(packed, struct):
    same_bytes(packed, struct)


def test_reached_from_the_package():
    """Next to the operators of their kind."""
    import test_sequence_layers_gb300 as ttt
    for n in ("ttt_rope_axes", "ttt_selective_scan_fwd", "ttt_selective_scan_bwd", "ttt_short_conv_fwd", "ttt_short_conv_bwd"):
        assert getattr(ttt, n) is getattr(abi, n)
    assert ttt.rope_axes is rotary.rope_axes and ttt.rope_axes_table is rotary.rope_axes_table


# ----------------------------------------------------------------------- convolution


def _conv_desc(**kw):
    d = dict(B=2, T=300, C=64, width=4, io_dtype=abi.TTT_BF16, act=1)
    strides = kw.pop("strides", None)
    d.update(kw)
    return abi.ShortConvDesc(*d.values(), (ctypes.c_longlong * 4)(*(strides or [d["T"] * d["C"], d["C"]] * 2)))


def _conv_fwd(L, x=_at(1), w=_at(2), bias=None, reset=None, state=None, y=_at(3), state_out=None, **kw):
    return L.ttt_short_conv_fwd(_conv_desc(**kw), x, w, bias, reset, state, y, state_out, None)


def _conv_bwd(L, dy=_at(1), x=_at(2), w=_at(3), bias=None, reset=None, state=None, dso=None, dx=_at(4), dw=_at(5), db=None,
              ds=None, ws=_at(6), nws=1 << 20, **kw):
    return L.ttt_short_conv_bwd(_conv_desc(**kw), dy, x, w, bias, reset, state, dso, dx, dw, db, ds, ws, ctypes.c_size_t(nws), None)


def test_conv_forward_refusals(L):
    assert L.ttt_short_conv_fwd(*[None] * 9) == -1
    for bad in (dict(B=-1), dict(T=-1), dict(C=0), dict(width=0), dict(act=2), dict(act=-1), dict(io_dtype=2), dict(x=None),
                dict(w=None), dict(y=None), dict(y=_at(1)), dict(y=_at(2)), dict(y=_at(1) + 64), dict(bias=_at(3)),
                dict(reset=_at(3)), dict(state=_at(3)), dict(state_out=_at(3)), dict(state_out=_at(1)),
                dict(state=_at(4), state_out=_at(4) + 16), dict(strides=[-1, 64, 0, 0])):
        assert _conv_fwd(L, **bad) == -1, bad
    assert _conv_fwd(L, width=5) == -2 and _conv_fwd(L, B=1 << 20, T=1 << 20) == -2
    assert _conv_fwd(L, C=(1 << 30) + 1) == -2
    assert _conv_fwd(L, B=0) == 0 and _conv_fwd(L, T=0) == 0
    for bad in (dict(x=_at(1) + 1), dict(y=_at(3) + 1), dict(w=_at(2) + 2), dict(bias=_at(5) + 1), dict(state=_at(5) + 1),
                dict(state_out=_at(5) + 1)):
        assert _conv_fwd(L, **bad) == -3, bad


def test_conv_backward_refusals(L):
    for bad in (dict(dy=None), dict(x=None), dict(dx=None), dict(w=None), dict(dx=_at(1)), dict(dx=_at(2)), dict(dw=_at(4)),
                dict(db=_at(5)), dict(ds=_at(4)), dict(ws=None), dict(nws=64), dict(ws=_at(4)), dict(dso=_at(4)), dict(T=-1)):
        assert _conv_bwd(L, **bad) == -1, bad
    for bad in (dict(dy=_at(1) + 1), dict(dx=_at(4) + 1), dict(dw=_at(5) + 2), dict(dso=_at(7) + 2), dict(ws=_at(6) + 4)):
        assert _conv_bwd(L, **bad) == -3, bad
    assert _conv_bwd(L, B=0, dw=None) == 0
    assert L.ttt_short_conv_bwd_workspace(None) == 0 and L.ttt_short_conv_bwd_workspace(_conv_desc(width=9)) == 0
    assert abi.ttt_short_conv_bwd_workspace(2, 300, 64, 4) >= 64 * 5 * 4


@pytest.mark.parametrize("over", [dict(B=1 << 20, T=1 << 20, C=8), dict(B=1, T=(1 << 31) - 1, C=8), dict(C=(1 << 30) + 1),
                                  dict(width=5), dict(B=1 << 16, T=1 << 15, C=8)])
def test_no_workspace_for_a_convolution_that_is_refused(L, over):
    """The binding allocates what the query says before the call can refuse."""
    assert _conv_bwd(L, **over) == -2 and _conv_fwd(L, **over) == -2
    assert L.ttt_short_conv_bwd_workspace(_conv_desc(**over)) == 0


@pytest.mark.parametrize("bad", [
    dict(x=_Dev((2, 9))), dict(x=_Dev((2, 9, 8), cuda=False)), dict(x=_Dev((2, 9, 8), torch.float16)),
    dict(x=_Dev((2, 9, 8), last=2)), dict(weight=_Dev((8, 4), BF)), dict(weight=_Dev((7, 4), F32)), dict(weight=_Dev((8,), F32)),
    dict(bias=_Dev((7,), F32)), dict(reset=_Dev((2, 8), torch.bool)), dict(state=_Dev((2, 3, 8), F32)),
    dict(state=_Dev((2, 4, 8))), dict(y=_Dev((2, 9, 9))), dict(state_out=_Dev((2, 2, 8))),
    dict(weight=_Dev((8, 4), F32, index=1)),
])
def test_conv_binding_refuses_before_any_launch(bad):
    a = dict(x=_Dev((2, 9, 8)), weight=_Dev((8, 4), F32), y=_Dev((2, 9, 8)))
    a.update(bad)
    with pytest.raises(ValueError):
        abi.ttt_short_conv_fwd(a.pop("x"), a.pop("weight"), **a)


# ------------------------------------------------------------------------------ scan


def _scan_desc(**kw):
    d = dict(B=2, T=300, C=64, N=16, G=1, io_dtype=abi.TTT_BF16, softplus=1)
    d.update(kw)
    tc, gn = d["C"], d["G"] * d["N"]
    s = [d["T"] * tc, tc] * 4 + [d["T"] * gn, gn, d["N"]] * 2
    return abi.ScanDesc(*d.values(), (ctypes.c_longlong * 14)(*s))


def _scan_fwd(L, A=_at(1), D=None, bias=None, x=_at(2), dl=_at(3), Bm=_at(4), Cm=_at(5), z=None, reset=None, h0=None, y=_at(6),
              h_last=None, states=None, ws=_at(7), nws=1 << 24, **kw):
    return L.ttt_selective_scan_fwd(_scan_desc(**kw), abi.ScanVectors(A, D, bias), x, dl, Bm, Cm, z, reset, h0, y, h_last,
                                    states, ws, ctypes.c_size_t(nws), None)


def _scan_bwd(L, A=_at(1), D=None, bias=None, dy=_at(2), x=_at(3), dl=_at(4), Bm=_at(5), Cm=_at(6), z=None, reset=None,
              states=_at(7), dhl=None, dx=_at(8), ddl=_at(9), dB=_at(10), dC=_at(11), dz=None, gA=_at(12), gD=None, gb=None,
              dh0=None, ws=_at(20), nws=1 << 26, **kw):
    return L.ttt_selective_scan_bwd(_scan_desc(**kw), abi.ScanVectors(A, D, bias), dy, x, dl, Bm, Cm, z, reset, states, dhl, dx,
                                    ddl, dB, dC, dz, abi.ScanVectors(gA, gD, gb), dh0, ws, ctypes.c_size_t(nws), None)


def test_scan_forward_refusals(L):
    assert L.ttt_selective_scan_fwd(*[None] * 13, 0, None) == -1
    assert L.ttt_selective_scan_fwd_workspace(_scan_desc()) > 0 and L.ttt_selective_scan_fwd_workspace(_scan_desc(T=1)) == 0
    for bad in (dict(B=-1), dict(T=-1), dict(C=0), dict(N=0), dict(G=0), dict(G=3), dict(softplus=2), dict(io_dtype=5), dict(A=None),
                dict(x=None), dict(dl=None), dict(Bm=None), dict(Cm=None), dict(y=None), dict(y=_at(2)), dict(y=_at(5)),
                dict(z=_at(6)), dict(h0=_at(6)), dict(h_last=_at(6)), dict(h0=_at(8), h_last=_at(8) + 16), dict(states=_at(6)),
                dict(states=_at(9), h0=_at(9)), dict(reset=_at(6)), dict(ws=None), dict(nws=128), dict(ws=_at(2)),
                dict(ws=_at(8), h0=_at(8)), dict(D=_at(6)), dict(h_last=_at(1))):
        assert _scan_fwd(L, **bad) == -1, bad
    for bad in (dict(N=65), dict(B=70000), dict(B=60000, T=1 << 20)):
        assert _scan_fwd(L, **bad) == -2, bad
    assert _scan_fwd(L, B=0) == 0 and _scan_fwd(L, T=0) == 0
    for bad in (dict(A=_at(1) + 2), dict(x=_at(2) + 1), dict(z=_at(8) + 1), dict(y=_at(6) + 1), dict(h0=_at(8) + 1),
                dict(states=_at(8) + 2), dict(bias=_at(8) + 3), dict(ws=_at(7) + 8)):
        assert _scan_fwd(L, **bad) == -3, bad


def test_scan_backward_refusals(L):
    assert L.ttt_selective_scan_bwd(*[None] * 19, 0, None) == -1
    for bad in (dict(dy=None), dict(x=None), dict(states=None), dict(dx=None), dict(ddl=None), dict(dB=None), dict(dC=None),
                dict(z=_at(13)), dict(dz=_at(13)), dict(gD=_at(13)), dict(gb=_at(13)), dict(ws=None), dict(nws=1024),
                dict(dx=_at(3)), dict(dx=_at(9)), dict(dB=_at(11)), dict(dh0=_at(8)), dict(dhl=_at(13), dh0=_at(13)),
                dict(ws=_at(7)), dict(gA=_at(1)), dict(C=-3)):
        assert _scan_bwd(L, **bad) == -1, bad
    for bad in (dict(dy=_at(2) + 1), dict(dB=_at(10) + 1), dict(states=_at(7) + 2), dict(gA=_at(12) + 1), dict(ws=_at(20) + 8)):
        assert _scan_bwd(L, **bad) == -3, bad
    assert _scan_bwd(L, N=80) == -2
    assert _scan_bwd(L, B=0, gA=None) == 0
    assert abi.ttt_selective_scan_bwd_workspace(2, 300, 64, 16) > 0 and abi.ttt_selective_scan_bwd_workspace(2, 300, 63, 16, 2) == 0


@pytest.mark.parametrize("bad", [
    dict(x=_Dev((2, 9))), dict(x=_Dev((2, 9, 8), cuda=False)), dict(x=_Dev((2, 9, 8), torch.float16)), dict(delta=_Dev((2, 9, 7))),
    dict(delta=_Dev((2, 9, 8), F32)), dict(A=_Dev((8, 16), BF)), dict(A=_Dev((16, 8), F32)), dict(A=_Dev((8,), F32)),
    dict(B=_Dev((2, 9, 15))), dict(B=_Dev((2, 9, 3, 16)), C=_Dev((2, 9, 3, 16))), dict(C=_Dev((2, 9, 2, 16))),
    dict(C=_Dev((2, 9, 16), last=2)), dict(D=_Dev((9,), F32)), dict(delta_bias=_Dev((8,), BF)), dict(z=_Dev((2, 9, 9))),
    dict(reset=_Dev((2, 9), F32)), dict(h0=_Dev((2, 8, 16), BF)), dict(h0=_Dev((2, 16, 8), F32)), dict(y=_Dev((2, 9, 8), F32)),
    dict(h_last=_Dev((1, 8, 16), F32)), dict(states=_Dev((2, 2, 8, 16), F32)), dict(x=_Dev((2, 9, 8), index=1)),
])
def test_scan_binding_refuses_before_any_launch(bad, monkeypatch):
    # (the parameters' addresses are packed with the descriptor, before the states are looked at)
    monkeypatch.setattr(_Dev, "data_ptr", lambda self: 1 << 20)
    monkeypatch.setattr(abi, "_call", lambda *a: pytest.fail("the binding reached the library with a bad argument"))
    a = dict(x=_Dev((2, 9, 8)), delta=_Dev((2, 9, 8)), A=_Dev((8, 16), F32), B=_Dev((2, 9, 16)), C=_Dev((2, 9, 16)),
             y=_Dev((2, 9, 8)), h_last=_Dev((2, 8, 16), F32), workspace=_Dev((1 << 20,), torch.uint8))
    a.update(bad)
    with pytest.raises(ValueError):
        abi.ttt_selective_scan_fwd(*[a.pop(n) for n in ("x", "delta", "A", "B", "C")], **a)


@pytest.mark.parametrize("st", [-1, 3])
def test_forward_passes_do_not_look_at_the_gradients_strides(L, st):
    """A description made for both directions: only the backward pass reads, and refuses, dy's."""
    conv, scan = _conv_desc(T=0, strides=[64, 64, st, st]), _scan_desc(T=0)
    scan.strides[6] = scan.strides[7] = st
    par = abi.ScanVectors(_at(1), None, None)
    assert L.ttt_short_conv_fwd(conv, _at(1), _at(2), None, None, None, _at(3), None, None) == 0
    assert L.ttt_selective_scan_fwd(scan, par, *[None] * 11, 0, None) == 0
    want = -1 if st < 0 else 0
    assert L.ttt_short_conv_bwd(conv, _at(1), _at(2), _at(3), *[None] * 4, _at(4), *[None] * 4, 0, None) == want
    assert L.ttt_selective_scan_bwd(scan, par, *[None] * 14, abi.ScanVectors(None, None, None), None, None, 0, None) == want


# --------------------------------------------------------------------------- streams


@pytest.fixture
def calls(gpu, monkeypatch):  # noqa: F811
    side, made, seen = gpu

    def entry(*args):
        seen.append(torch.cuda.current_stream().name)
        return 0
    for n in ("ttt_rope_axes", "ttt_short_conv_fwd", "ttt_short_conv_bwd", "ttt_selective_scan_fwd", "ttt_selective_scan_bwd"):
        monkeypatch.setitem(abi._fns, n, entry)
    monkeypatch.setattr(abi, "_workspace_bytes", lambda name, desc: 4096)
    return gpu


def test_streams(calls):
    side, made, seen = calls
    x, w = _T((2, 9, 8)), _T((8, 4), F32)
    A, B, C = _T((8, 16), F32), _T((2, 9, 16)), _T((2, 9, 16))
    h, st = _T((2, 8, 16), F32), _T((2, 1, 8, 16), F32)
    # everything allocated, and what of it is returned to the current stream
    for n, back, fn, args, kw in (
            (2, 2, abi.ttt_short_conv_fwd, (x, w), dict(want_state=True)),
            (3, 2, abi.ttt_short_conv_bwd, (x, x, w), {}),
            (4, 3, abi.ttt_selective_scan_fwd, (x, x, A, B, C), dict(h0=h, want_states=True)),
            (7, 6, abi.ttt_selective_scan_bwd, (x, x, x, A, B, C, st), {}),
            (1, 1, abi.ttt_rope_axes, (_T((2, 3, 4, 16)), None, None, _T((9, 8, 2), F32), bytes(8)), dict(grid=(2, 2)))):
        made.clear(), seen.clear()
        got = _check(calls, fn, *args, **kw)
        assert len(got) == n and sum("current" in t.used_on for t in got) == back, fn.__name__
