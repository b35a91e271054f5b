"""The stream= argument of the binding, without a GPU: what a call allocates belongs to
the given stream, its inputs are kept for that stream's work, and its results for the work
of the stream that was current."""
import contextlib

import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests.test_rotary import _Dev

BF, F32 = torch.bfloat16, torch.float32


class _T(_Dev):
    """A device tensor without a device; knows the stream that it was allocated on."""

    def __init__(self, shape, dtype=BF, owner=None):
        super().__init__(shape, dtype)
        self.owner, self.used_on = owner, set()

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        self.used_on.add(stream.name)


class _Stream:
    device, cuda_stream = torch.device("cuda", 0), 77

    def __init__(self, name):
        self.name = name


@pytest.fixture
def gpu(monkeypatch):
    """Streams and allocations without a GPU; returns the side stream, the tensors
    allocated, and the stream of every library call."""
    current, side = _Stream("current"), _Stream("side")
    active, made, calls = [current], [], []

    @contextlib.contextmanager
    def use(stream):
        active.append(stream)
        yield
        active.pop()

    def empty(*shape, dtype=F32, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        made.append(_T(shape, dtype, active[-1].name))
        return made[-1]

    def entry(*args):
        calls.append(active[-1].name)
        return 0
    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: active[-1])
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(abi, "_empty", empty)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape, dtype=t.dtype))
    monkeypatch.setattr(abi, "_raw_stream", lambda di: 0)
    monkeypatch.setattr(abi, "_current_device", lambda: 0)
    monkeypatch.setattr(abi, "_norm_workspace", lambda desc: 4096)
    monkeypatch.setattr(abi, "_fns", {n: entry for n in ("ttt_rope", "ttt_block_norm_fwd", "ttt_block_norm_bwd",
                                                         "ttt_recurrence_fwd", "ttt_recurrence_bwd")})
    return side, made, calls


def _check(gpu, fn, *args, **kw):
    side, made, calls = gpu
    fn(*args, stream=side, **kw)
    assert made and all(t.owner == "side" for t in made), [t.owner for t in made]
    assert calls == ["side"]
    for t in (*args, *kw.values()):
        if isinstance(t, _T):
            assert "side" in t.used_on
    return made


def test_rope(gpu):
    q, k, v = (_T((2, 3, 4, 16)) for _ in range(3))
    made = _check(gpu, abi.ttt_rope, q, k, v, _T((9, 8, 2), F32), positions=_T((2, 4), torch.int64))
    assert len(made) == 3 and all("current" in t.used_on for t in made)


def test_block_norm(gpu):
    y, x, g, w = _T((2, 4, 64)), _T((2, 4, 64)), _T((2, 4, 64)), _T((64,), F32)
    made = _check(gpu, abi.ttt_block_norm_fwd, y, x=x, gate=g, post="rms", post_weight=w, pre="rms", want_stats=True)
    assert len(made) == 3 and all("current" in t.used_on for t in made)


def test_block_norm_backward(gpu):
    y, x, g, w = _T((2, 4, 64)), _T((2, 4, 64)), _T((2, 4, 64)), _T((64,), F32)
    made = _check(gpu, abi.ttt_block_norm_bwd, _T((2, 4, 64)), _T((2, 4, 64)), y, _T((2, 4, 4), F32), x=x, gate=g,
                  post="rms", post_weight=w, pre="rms")
    assert len(made) == 5  # dy, dx, dgate, the weight's gradient and the workspace
    assert sum("current" in t.used_on for t in made) == 4


def test_recurrence(gpu):
    x, f, h0 = _T((2, 9, 8)), _T((2, 9, 8)), _T((2, 8), F32)
    assert len(_check(gpu, abi.ttt_recurrence_fwd, x, f, h0, want_states=True)) == 3


def test_recurrence_backward(gpu):
    x, f, dh = _T((2, 9, 8)), _T((2, 9, 8)), _T((2, 9, 8))
    assert len(_check(gpu, abi.ttt_recurrence_bwd, dh, x, f, _T((2, 1, 8), F32))) == 3


def _library(monkeypatch, gpu):
    side, made, calls = gpu

    class Lib:
        def __getattr__(self, name):
            if name.endswith("workspace"):
                return lambda *a: 4096
            return lambda *a: calls.append(torch.cuda.current_stream().name) or 0
    monkeypatch.setattr(abi, "lib", Lib)


def test_linear(gpu, monkeypatch):
    _library(monkeypatch, gpu)
    q, W = _T((2, 3, 256, 64)), _T((3, 64, 64), F32)
    assert len(_check(gpu, abi.ttt_linear_fwd, q, q, q, W, 16, eta=_T((2, 3, 256), F32))) == 2


def test_linear_seqpar_workspace(gpu, monkeypatch):
    _library(monkeypatch, gpu)
    q, W = _T((2, 3, 256, 64)), _T((3, 64, 64), F32)
    made = _check(gpu, abi.ttt_linear_fwd_seqpar, q, q, q, W, 16)
    assert len(made) == 3 and sum("current" in t.used_on for t in made) == 2


def test_mlp(gpu, monkeypatch):
    _library(monkeypatch, gpu)
    q = _T((2, 3, 256, 64))
    P = [_T(s, F32) for s in ((3, 64, 256), (3, 256), (3, 256, 64), (3, 64))]
    made = _check(gpu, abi.ttt_mlp_fwd, q, q, q, *P, 16)
    assert len(made) == 5 and all("current" in t.used_on for t in made)


def test_dwconv_and_gate(gpu, monkeypatch):
    _library(monkeypatch, gpu)
    q = _T((1, 2, 196, 64))
    assert len(_check(gpu, abi.ttt_dwconv_fwd, q, q, q, _T((2, 9, 64), F32), 14, 14)) == 2
    gpu[1].clear(), gpu[2].clear()
    assert len(_check(gpu, abi.ttt_eta_gate, _T((2, 50, 256)), _T((4, 256)))) == 1


def test_a_stream_of_another_device_is_refused(gpu):
    side, made, calls = gpu
    side.device = torch.device("cuda", 1)
    with pytest.raises(ValueError):
        abi.ttt_rope(_T((2, 3, 4, 16)), None, None, _T((9, 8, 2), F32), stream=side)
    assert not made and not calls
