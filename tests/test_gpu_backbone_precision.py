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


def _first_state(B, T, N):
    """B or C with ones in their first state alone."""
    m = torch.zeros(B, T, N, device="cuda")
    m[..., 0] = 1
    return m


# single tokens, rows of single elements, of 16 bytes, pieces, whole sequences
SHAPES = [(2, 1, 96), (2, 40, 37), (1, 40, 96), (1, 300, 64), (24, 75, 1056)]


@pytest.mark.parametrize("B,T,C", SHAPES)
def test_gate_of_the_scan(B, T, C):
    """With B zero, D and x one the output before the gate is one."""
    N, n = 16, B * T * C
    x, A, zero = torch.ones(B, T, C, device="cuda"), -torch.ones(C, N, device="cuda"), torch.zeros(B, T, N, device="cuda")
    D = torch.ones(C, device="cuda")
    z = torch.linspace(-80, 80, n, device="cuda").view(B, T, C)
    y = abi.ttt_selective_scan_fwd(x, x, A, zero, zero, D=D, z=z)[0]
    _within("y", y, _silu(z.double()), z, 2.0 ** -21)
    z = -2 - 78 * torch.rand(B, T, C, device="cuda")
    states = abi.ttt_selective_scan_fwd(x, x, A, zero, zero, D=D, z=z, want_states=True)[2]
    dz = abi.ttt_selective_scan_bwd(x, x, x, A, zero, zero, states, D=D, z=z).z
    _within("dz", dz, _slope(z.double()), z, 2.0 ** -20)
    abi.ttt_sync_status()


@pytest.mark.parametrize("B,T,C", SHAPES)
def test_rate_of_the_scan(B, T, C):
    """With a reset at every token, one state and x one the output is the rate."""
    N, n = 16, B * T * C
    x, A, one = torch.ones(B, T, C, device="cuda"), -torch.ones(C, N, device="cuda"), _first_state(B, T, N)
    reset = torch.ones(B, T, dtype=torch.bool, device="cuda")
    delta = torch.linspace(-80, 25, n, device="cuda").view(B, T, C)
    y, _, states = abi.ttt_selective_scan_fwd(x, delta, A, one, one, reset=reset, want_states=True)
    v = delta.double()
    _within("rate", y, v.clamp(min=0) + torch.log1p(torch.exp(-v.abs())), delta, 2.0 ** -21)
    slope = abi.ttt_selective_scan_bwd(x, x, delta, A, one, one, states, reset=reset).delta
    _within("slope", slope, torch.sigmoid(v), delta, 2.0 ** -21)
    abi.ttt_sync_status()


@pytest.mark.parametrize("B,T,C", [(64, 8, 512), (8, 64, 512), (24, 64, 1056)])  # few tokens, tiles, whole sequences
@pytest.mark.parametrize("lo,hi", [(0.001, 0.01), (0.01, 0.1), (0.1, 0.5)])
def test_decays_have_no_mean_error(B, T, C, lo, hi):
    """States that only decay: the mean over all of them, per token, of the relative error.  The
    kernels' decays claim 9e-9, below 2^-26; 2^-24 sqrt(T) of rounding in each state averages to below 2^-30
    over 2^18 of them and more."""
    N = 16
    g = torch.Generator(device="cuda").manual_seed(7)
    d = 0.6 + 0.8 * torch.rand(B, T, C, device="cuda", generator=g)
    A = -(lo + (hi - lo) * torch.rand(C, N, device="cuda", generator=g))
    zero, zbc = torch.zeros(B, T, C, device="cuda"), torch.zeros(B, T, N, device="cuda")
    h0 = 1 + torch.rand(B, C, N, device="cuda", generator=g)
    last = abi.ttt_selective_scan_fwd(zero, d, A, zbc, zbc, softplus=False, h0=h0)[1]
    abi.ttt_sync_status()
    want = h0.double() * torch.exp(d.double().sum(1)[..., None] * A.double())
    err = (last.double() - want) / want
    assert abs(float(err.mean())) <= T * 2.0 ** -26, float(err.mean()) / T
