"""SiLU, softplus and their slopes of fp32 tensors in the short convolution and the selective
scan, entry by entry relative to themselves.  From the arithmetic, in units of 2^-24: an exponential
2, 1 + e 1, its reciprocal 2, a product or sum 1.  silu(v) = v / (1 + exp(-v)): 6.  Its slope
s (1 + v (1 - s)) for v <= -2, where |v| / |1 + v| <= 2: s 5, 1 - s 2 of the sum, the sum 1, products
1 each, at most four: 12.  softplus(v) = log(1 + e), e = exp(v), for v <= 0: e 2, the polynomial 4, a
product 1; for v > 0 a sum more, of smaller terms.  Its slope e / (1 + e): 6, and a product by the
gradient."""
import pytest
import torch

from test_sequence_layers_gb300 import abi
from tests import gpu_common as G

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def _within(name, got, want, at, bound):
    err = ((got.double() - want) / want).abs().flatten()
    assert float(err.max()) <= bound, (name, float(err.max()) / bound, float(at.flatten()[err.argmax()]))


def _silu(v):
    return v * torch.sigmoid(v)


def _slope(v):
    s = torch.sigmoid(v)
    return s * (1 + v * torch.sigmoid(-v))


@pytest.mark.parametrize("C", [512, 501, 502])  # four channels a thread, one, two
@pytest.mark.parametrize("T", [1, 40])
def test_convolution(T, C):
    """One tap of weight one: y is the activation of x itself, dx its slope."""
    x = torch.linspace(-80, 80, T * C, device="cuda").view(1, T, C)
    one = torch.ones(C, 1, device="cuda")
    y, _ = abi.ttt_short_conv_fwd(x, one)
    _within("y", y, _silu(x.double()), x, 2.0 ** -21)
    x = -2 - 78 * torch.rand(1, T, C, device="cuda")
    dx = abi.ttt_short_conv_bwd(torch.ones_like(x), x, one).x
    _within("dx", dx, _slope(x.double()), x, 2.0 ** -20)
    abi.ttt_sync_status()
