"""Host threads, each on a stream of its own, launching the same kernels with other amounts
of shared memory: no launch is refused and every result is the one of a single thread.  The
library's own calls are repeated with the arguments that the binding made, so that the
threads spend their time inside the library, where they run side by side."""
import threading

import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROUNDS = 3000


class _Recorded:
    """A library call (its last argument the stream), its outputs and what it points to."""

    def __init__(self, monkeypatch, wrapper, *args, **kw):
        self.kept = (args, kw)
        with monkeypatch.context() as m:
            real = abi.lib()

            class Lib:
                def __getitem__(_, name):
                    return real[name]

                def __getattr__(_, name):
                    if name.endswith(("workspace", "str")):
                        return getattr(real, name)

                    def record(*a):
                        self.fn, self.args = getattr(real, name), a[:-1]
                        return 0
                    return record

            def call(name, di, *a):
                self.fn, self.args = abi._fn(name), a
            m.setattr(abi, "lib", Lib)
            m.setattr(abi, "_call", call)
            out = wrapper(*args, **kw)
        self.out = [t for t in out if t is not None]
        torch.cuda.synchronize()

    def run(self, rounds, stream):
        for _ in range(rounds):
            rc = self.fn(*self.args, stream)
            if rc != 0:
                raise abi.TTTError("a thread's call", rc)


def _in_threads(calls):
    torch.cuda.synchronize()
    for c in calls:
        c.run(1, torch.cuda.current_stream().cuda_stream)
    abi.ttt_sync_status()
    want = [[t.clone() for t in c.out] for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(calls))

    def work(call, st):
        try:
            with torch.cuda.device(0):
                start.wait()
                for _ in range(10):
                    call.run(ROUNDS // 10, st.cuda_stream)
                    st.synchronize()
        except Exception as e:  # reported by the test's own thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    abi.ttt_sync_status()
    torch.cuda.synchronize()
    for c, ref in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(c.out, ref))


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def test_block_norm_backward_of_two_widths(monkeypatch):
    def call(D):
        y, g, dh, du = (torch.randn(1, 20, D, device="cuda").to(BF) for _ in range(4))
        kw = dict(gate=g, act="silu", post="rms", post_weight=torch.randn(D, device="cuda"), pre="rms")
        _, _, st = abi.ttt_block_norm_fwd(y, want_stats=True, **kw)
        ws = torch.empty(abi.ttt_block_norm_bwd_workspace(1, 20, D), dtype=torch.uint8, device="cuda")
        return _Recorded(monkeypatch, abi.ttt_block_norm_bwd, dh, du, y, st, workspace=ws, **kw)
    _in_threads([call(4096), call(2048)])


def test_recurrence_of_two_shapes(monkeypatch):
    def call(B, T, C):
        x, f = (torch.randn(B, T, C, device="cuda").to(BF) for _ in range(2))
        return _Recorded(monkeypatch, abi.ttt_recurrence_fwd, x, f)
    _in_threads([call(1, 2048, 64), call(1, 128, 64)])


@pytest.mark.parametrize("kind", ["linear_f32", "mlp_f32", "full_batch", "dwconv"])
def test_layer_of_two_shapes(kind, monkeypatch):
    def call(n):
        r = lambda *s: 0.1 * torch.randn(*s, device="cuda")
        if kind == "linear_f32":
            d = (128, 32)[n]
            q, W = r(1, 2, 16, d), r(2, d, d)
            return _Recorded(monkeypatch, abi.ttt_linear_fwd, q, q, q, W, 16)
        if kind == "mlp_f32":
            d, m = ((64, 128), (32, 64))[n]
            q, P = r(1, 2, 16, d), (r(2, d, m), r(2, m), r(2, m, d), r(2, d))
            return _Recorded(monkeypatch, abi.ttt_mlp_fwd, q, q, q, *P, 16, want_W=False)
        if kind == "full_batch":
            T = (256, 64)[n]
            q, W = r(1, 2, T, 64).to(BF), r(2, 64, 64)
            return _Recorded(monkeypatch, abi.ttt_linear_fwd, q, q, q, W, T, causal=False, epochs=2)
        N = (14, 8)[n]
        q, W = r(1, 2, N * N, 64).to(BF), r(2, 9, 64)
        return _Recorded(monkeypatch, abi.ttt_dwconv_fwd, q, q, q, W, N, N)
    _in_threads([call(0), call(1)])
