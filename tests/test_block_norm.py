"""Refusals of the block norm at the C boundary and in the binding, without a GPU."""
import ctypes

import pytest
import torch

from test_sequence_layers_gb300 import abi, build
from tests.test_rotary import _Dev

FAKE = 1 << 20
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    build.build()
    return abi.lib()


def _desc(**kw):
    d = dict(B=2, T=4, D=64, heads=1, io_dtype=abi.TTT_BF16, post=1, pre=2, act=2, post_eps=1e-6, pre_eps=1e-6,
             alpha=1.0)
    d.update(kw)
    st = [d["T"] * d["D"], 0 if d["heads"] == 1 else d["T"] * d["D"] // max(1, d["heads"]), d["D"] // max(1, d["heads"])]
    return abi.BlockNormDesc(*d.values(), (ctypes.c_longlong * 11)(*st, *([d["T"] * d["D"], d["D"]] * 4)))


def _at(i):
    return FAKE + i * (1 << 24)


def _fwd(L, par=(), y=_at(1), x=_at(2), g=_at(3), h=_at(4), u=_at(5), stats=None, **kw):
    p = abi.BlockNormVectors(**dict(par))
    return L.ttt_block_norm_fwd(_desc(**kw), p, y, x, g, h, u, stats, None)


def _bwd(L, par=(), grads=(), dh=_at(1), du=_at(2), y=_at(3), x=_at(4), g=_at(5), stats=_at(6), dy=_at(7), dx=_at(8),
         dg=_at(9), ws=_at(10), nws=1 << 23, **kw):
    return L.ttt_block_norm_bwd(_desc(**kw), abi.BlockNormVectors(**dict(par)), dh, du, y, x, g, stats, dy, dx, dg,
                                abi.BlockNormVectors(**dict(grads)), ws, nws, None)


def test_forward_refusals(L):
    assert L.ttt_block_norm_fwd(None, None, None, None, None, None, None, None, None) == -1
    for bad in (dict(B=-1), dict(T=-2), dict(D=0), dict(heads=0), dict(heads=3), dict(io_dtype=4), dict(post=3),
                dict(pre=-1), dict(act=4), dict(post_eps=-1.0), dict(pre_eps=float("nan")), dict(y=None), dict(g=None),
                dict(act=0), dict(h=None), dict(u=None), dict(pre=0), dict(par=dict(post_bias=_at(8))),
                dict(pre=0, u=None, par=dict(pre_weight=_at(8))), dict(h=_at(1)), dict(h=_at(2) + 64), dict(u=_at(2)),
                dict(u=_at(4)), dict(stats=_at(3))):
        assert _fwd(L, **bad) == -1, bad
    assert _fwd(L, D=8193) == -2
    assert _fwd(L, B=0) == 0 and _fwd(L, T=0) == 0
    for bad in (dict(y=_at(1) + 1), dict(h=_at(4) + 1), dict(stats=_at(6) + 8), dict(par=dict(scale=_at(8) + 2))):
        assert _fwd(L, **bad) == -3, bad


def test_backward_refusals(L):
    for bad in (dict(dy=None), dict(stats=None), dict(du=None), dict(pre=0), dict(dg=None), dict(x=None), dict(dh=None,
                du=None, pre=0), dict(grads=dict(post_bias=_at(11))), dict(grads=dict(scale=_at(11))),
                dict(grads=dict(post_weight=_at(11)), ws=None), dict(grads=dict(post_weight=_at(11)), nws=16),
                dict(dy=_at(3)), dict(dx=_at(9)), dict(dx=_at(1) + 32),
                dict(grads=dict(post_weight=_at(11), pre_weight=_at(11)))):
        assert _bwd(L, **bad) == -1, bad
    assert _bwd(L, stats=_at(6) + 4) == -3
    assert _bwd(L, grads=dict(post_weight=_at(11)), ws=_at(10) + 4) == -3
    assert _bwd(L, T=0) == 0


def test_workspace_holds_the_partial_sums(L):
    assert L.ttt_block_norm_bwd_workspace(None) == 0
    assert L.ttt_block_norm_bwd_workspace(_desc(D=9000)) == 0
    assert L.ttt_block_norm_bwd_workspace(_desc(T=0)) == 0
    assert abi.ttt_block_norm_bwd_workspace(1, 1, 768) == 5 * 768 * 4
    assert abi.ttt_block_norm_bwd_workspace(8, 2048, 768) >= 152 * 5 * 768 * 4


@pytest.mark.parametrize("bad", [
    dict(y=_Dev((2, 4))), dict(y=_Dev((2, 4, 64), cuda=False)), dict(y=_Dev((2, 4, 64), torch.float16)),
    dict(y=_Dev((2, 4, 64), last=2)), dict(x=_Dev((2, 4, 32))), dict(x=_Dev((2, 4, 64), F32)), dict(gate=None, act="silu"),
    dict(act="none"), dict(scale=_Dev((63,), F32)), dict(scale=_Dev((64,), BF)), dict(pre="none", u=_Dev((2, 4, 64))),
    dict(h=_Dev((2, 4, 63))), dict(stats=_Dev((2, 4, 3), F32)), dict(post_weight=_Dev((64,), F32, index=1)),
])
def test_binding_refuses_before_any_launch(bad):
    a = dict(y=_Dev((2, 4, 64)), x=_Dev((2, 4, 64)), gate=_Dev((2, 4, 64)), h=_Dev((2, 4, 64)), u=_Dev((2, 4, 64)),
             pre="rms", stats=_Dev((2, 4, 4), F32))
    a.update(bad)
    if a["pre"] == "none" and "u" not in bad:
        a["u"] = None
    with pytest.raises(ValueError):
        abi.ttt_block_norm_fwd(a.pop("y"), **a)
