"""A host thread whose first CUDA work of any kind is a call of this library: entry points
that make TMA descriptors work there as on any other thread."""
import threading

import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import gpu_common as G
from tests.test_gpu_threads import _Recorded

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("kind", ["linear", "linear_full_batch", "mlp", "gate", "dwconv", "recurrence"])
def test_first_call_of_a_thread(kind, monkeypatch):
    G.ensure_built()
    r = lambda *s: 0.1 * torch.randn(*s, device="cuda")
    q = r(1, 2, 196, 64).to(BF)
    if kind == "linear":
        c = _Recorded(monkeypatch, abi.ttt_linear_fwd, q, q, q, r(2, 64, 64), 16)
    elif kind == "linear_full_batch":
        c = _Recorded(monkeypatch, abi.ttt_linear_fwd, q, q, q, r(2, 64, 64), 196, causal=False)
    elif kind == "mlp":
        P = (r(2, 64, 256), r(2, 256), r(2, 256, 64), r(2, 64))
        c = _Recorded(monkeypatch, abi.ttt_mlp_fwd, q, q, q, *P, 16, eta_scalar=0.001, want_W=False)
    elif kind == "gate":
        eta = torch.empty(2, 4, 50, device="cuda")
        c = _Recorded(monkeypatch, abi.ttt_eta_gate, r(2, 50, 256).to(BF), r(4, 256).to(BF), eta=eta)
        c.out = [eta]
    elif kind == "dwconv":
        c = _Recorded(monkeypatch, abi.ttt_dwconv_fwd, q, q, q, r(2, 9, 64), 14, 14)
    else:
        c = _Recorded(monkeypatch, abi.ttt_recurrence_fwd, r(2, 300, 64).to(BF), r(2, 300, 64).to(BF))
    stream = torch.cuda.current_stream().cuda_stream
    c.run(1, stream)
    abi.ttt_sync_status()
    want = [t.clone() for t in c.out]
    for t in c.out:
        t.zero_()
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            c.run(1, stream)
        except Exception as e:  # reported by the test's own thread
            errors.append(e)
    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not errors, errors
    abi.ttt_sync_status()
    assert all(torch.equal(a, b) for a, b in zip(c.out, want))
