"""Paths of the short convolution and the selective scan that only some sizes and alignments
reach: whole sequences with rows that are not aligned, backward pieces of several tiles with more
than 16 states, resets and gradients at such sizes, more threads than 32 bits count."""
import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import backbone_defs as D
from tests import gpu_common as G
from tests.test_gpu_backbone import _room  # noqa: F401
from tests.test_gpu_selective_scan import _check, _run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _odd(t):
    """The same values one element past a 16-byte boundary, rows an odd stride apart."""
    flat = t.flatten(2)
    wide = torch.full((*flat.shape[:2], flat.shape[2] + 6 - flat.shape[2] % 2 + 1), 5.0, device=t.device, dtype=t.dtype)
    wide[..., 1:1 + flat.shape[2]] = flat
    return wide[..., 1:1 + flat.shape[2]].unflatten(-1, t.shape[2:])


def _unaligned(i, names):
    j = dict(i, **{n: _odd(i[n]) for n in names if i[n] is not None})
    assert all(j[n].stride(1) % 2 and j[n].data_ptr() % 16 for n in names if i[n] is not None)
    return j


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [8, 16])
@pytest.mark.parametrize("names", [("B", "C"), ("x",), ("x", "delta", "z", "B", "C", "dy")])
@pytest.mark.parametrize("resets", [0.0, 0.05])
def test_whole_sequences_of_unaligned_rows(N, names, resets, dtype):
    """B and C behind an odd rank in their projection; gradients too, with resets."""
    # (792 warps of the tile kernel would cut a long sequence)
    assert abi.ttt_selective_scan_fwd_workspace(24, 4096, 1056, N, 2) == 0
    i = D.scan_inputs(24, 75, 1056, N, 2, dtype=dtype, resets=resets, seed=N)
    _check(_unaligned(i, names))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [8, 16])
@pytest.mark.parametrize("resets", [0.0, 0.05])
def test_whole_sequences_of_aligned_rows(N, resets, dtype):
    _check(D.scan_inputs(24, 75, 1056, N, 2, dtype=dtype, resets=resets, seed=3))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [20, 24, 40, 64])
@pytest.mark.parametrize("resets", [0.0, 0.1])
@pytest.mark.parametrize("odd", [False, True])
def test_pieces_of_two_tiles(N, resets, odd, dtype):
    """Two chunks are never cut: one block takes both tiles, the second one not full."""
    i = D.scan_inputs(2, 61, 72, N, 2, dtype=dtype, resets=resets, seed=N)
    _check(_unaligned(i, ("x", "delta", "z", "B", "C", "dy")) if odd else i)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,B,resets", [(24, 20, 0.0), (24, 20, 0.05), (64, 10, 0.0), (64, 10, 0.05)])
def test_pieces_of_many_tiles(N, B, resets, dtype):
    """Enough channels that a sequence of five tiles is one piece."""
    _check(D.scan_inputs(B, 150, 512, N, dtype=dtype, resets=resets, seed=N))


def test_many_tiles_twice_give_the_same_bits():
    i = D.scan_inputs(20, 150, 512, 24, resets=0.05)
    one, two = _run(i), _run(i)
    assert all(torch.equal(one[n], two[n]) for n in one)


def test_more_threads_than_32_bits_count(_room):  # noqa: F811
    """Single tokens of 2^23 + 3 sequences: 2^31 threads of four channels and more."""
    B, C, tail = (1 << 23) + 3, 1024, 5
    x = torch.empty(B, 1, C, device="cuda", dtype=BF).normal_()
    w, b = torch.randn(C, 4, device="cuda"), torch.randn(C, device="cuda")
    y, _ = abi.ttt_short_conv_fwd(x, w, b)
    for at in (slice(0, tail), slice(B // 2, B // 2 + tail), slice(B - tail, B)):
        assert torch.equal(y[at], abi.ttt_short_conv_fwd(x[at].contiguous(), w, b)[0])
    abi.ttt_sync_status()
