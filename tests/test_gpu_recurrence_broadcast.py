"""The recurrence on inputs broadcast along time whose rows begin at any element: tokens
past the end read as zeros, whatever the shared memory held before (a pass over NaNs runs
first).  Tolerances as for the other sizes (fp32 2^-13, bf16 outputs 2^-8 of the largest
entry or one)."""
import numpy as np
import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import gpu_common as G
from tests.test_gpu_recurrence import TOL, _inputs, _loop

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,C", [(150, 64), (150, 7), (33, 129), (1000, 66)])
def test_inputs_broadcast_along_time(T, C, dtype):
    B = 2
    base = _inputs(B, 1, C, "mix", dtype, seed=T + C)

    def expanded(t, off):
        flat = torch.full((B * C + 16,), float("nan"), device="cuda", dtype=dtype)[off:off + B * C]
        flat.copy_(t.flatten())
        return flat.view(B, 1, C).expand(B, T, C)
    dirty = torch.full((B, T, C + 1), float("nan"), device="cuda", dtype=dtype)[..., 1:]
    _, _, st = abi.ttt_recurrence_fwd(dirty, dirty, want_states=True)
    i = dict(base, **{k: expanded(base[k], 0).contiguous() for k in ("x", "f", "dh")})
    want = _loop(i, "mix")
    for off in range(16 // base["x"].element_size()):
        j = {k: expanded(base[k], (off + s) % 8) for s, k in enumerate(("x", "f", "dh"))}
        abi.ttt_recurrence_bwd(dirty, dirty, dirty, st)
        h, hl, states = abi.ttt_recurrence_fwd(j["x"], j["f"], base["h0"], want_states=True)
        abi.ttt_recurrence_bwd(dirty, dirty, dirty, st)
        dx, df, dh0 = abi.ttt_recurrence_bwd(j["dh"], j["x"], j["f"], states, dh_last=base["dh_last"])
        abi.ttt_sync_status()
        for name, a, b in zip(("h", "h_last", "dx", "df", "dh0"), (h, hl, dx, df, dh0), want):
            a, e = a.double().cpu().numpy(), TOL[a.dtype]
            assert np.isfinite(a).all(), (name, off)
            assert np.abs(a - b).max() <= e * max(1.0, np.abs(b).max()), (name, off)
