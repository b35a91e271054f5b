"""The 64-bit token loops that the GPU tests of the short convolution and the selective scan
compare with: against independent forms (a library convolution, one packed sequence at a
time), their gradients against differentiation and against central differences."""
import pytest
import torch

from tests import backbone_defs as D

F64 = torch.float64


def _f64(i):
    return {k: t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t for k, t in i.items()}


@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_conv_is_the_library_convolution(K, act):
    i = _f64(D.conv_inputs(2, 9, 5, K, act=act, device="cpu"))
    got = D.conv(i)
    rows = torch.cat([i["state"], i["x"]], 1).transpose(1, 2)
    want = torch.nn.functional.conv1d(rows, i["weight"][:, None], i["bias"], groups=5).transpose(1, 2)
    if act == "silu":
        want = torch.nn.functional.silu(want)
    assert torch.allclose(got["y"][0], want, rtol=0, atol=1e-13)
    assert torch.equal(got["state_out"][0], rows.transpose(1, 2)[:, 9:])


def test_conv_of_packed_sequences_is_each_by_itself():
    i = _f64(D.conv_inputs(1, 12, 3, 4, device="cpu"))
    i["reset"] = torch.zeros(1, 12, dtype=torch.bool)
    i["reset"][0, [5, 6]] = True
    i["x"][0, 4] = float("inf")  # seen by no later sequence
    got = D.conv(i)["y"][0]
    for lo, hi, state in ((0, 4, i["state"]), (5, 6, None), (6, 12, None)):
        part = dict(i, x=i["x"][:, lo:hi], state=state, reset=None, dy=None)
        assert torch.allclose(got[:, lo:hi], D.conv(part)["y"][0], rtol=0, atol=1e-13)


def _grads_against_autograd(i, fn, leaves, outs, names):
    i = _f64(i)
    for n in leaves:
        if i[n] is not None:
            i[n].requires_grad_()
    got = fn(i)
    loss = sum((got[o][0] * i[d]).sum() for o, d in outs if i[d] is not None)
    present = [n for n in leaves if i[n] is not None]
    grads = torch.autograd.grad(loss, [i[n] for n in present], allow_unused=True)
    for n, g in zip(present, grads):
        want = torch.zeros_like(i[n]) if g is None else g
        assert torch.allclose(got[names[n]][0], want, rtol=1e-10, atol=1e-10), n
    # along one direction, by central differences of the forward values
    torch.manual_seed(1)
    for n, g in zip(present, grads):
        if g is None:
            continue
        v, eps, vals = torch.randn_like(i[n]), 1e-6, []
        for sign in (1, -1):
            j = {k: t.detach() if isinstance(t, torch.Tensor) else t for k, t in i.items()}
            j[n] = j[n] + sign * eps * v
            f = fn(j)
            vals.append(float(sum((f[o][0] * j[d]).sum() for o, d in outs if j[d] is not None)))
        slope = (vals[0] - vals[1]) / (2 * eps)
        # rounding 2^-52 of the values over eps, and eps^2 of the third derivative
        assert abs(slope - float((g * v).sum())) <= 1e-6 * (1 + abs(slope)), n


@pytest.mark.parametrize("kw", [dict(K=4), dict(K=3, act="none", resets=0.2), dict(K=2, state=False, bias=False),
                                dict(K=4, resets=0.3), dict(K=4, T=2)])
def test_conv_gradients(kw):
    i = D.conv_inputs(2, kw.pop("T", 11), 3, kw.pop("K"), device="cpu", **kw)
    _grads_against_autograd(i, D.conv, ("x", "weight", "bias", "state"), (("y", "dy"), ("state_out", "dstate_out")),
                            dict(x="dx", weight="dweight", bias="dbias", state="dstate"))


@pytest.mark.parametrize("kw", [dict(), dict(G=2, resets=0.2), dict(softplus=False, gate=False), dict(skip=False, state=False),
                                dict(T=1)])
def test_scan_gradients(kw):
    i = D.scan_inputs(2, kw.pop("T", 9), 4, 3, device="cpu", **kw)
    _grads_against_autograd(i, D.scan, ("x", "delta", "A", "B", "C", "D", "z", "delta_bias", "h0"),
                            (("y", "dy"), ("h_last", "dh_last")),
                            dict(x="dx", delta="ddelta", A="dA", B="dB", C="dC", D="dD", z="dz", delta_bias="ddelta_bias", h0="dh0"))


def test_scan_of_one_state_and_rate_one_is_a_sum():
    """A = 0: nothing decays, so y_t = C_t sum_{s <= t} x_s B_s from each sequence's start on."""
    i = _f64(D.scan_inputs(1, 8, 1, 1, softplus=False, gate=False, skip=False, state=False, train=False, device="cpu"))
    i["A"], i["delta"] = torch.zeros(1, 1, dtype=F64), torch.ones(1, 8, 1, dtype=F64)
    i["reset"] = torch.tensor([[0, 0, 0, 1, 0, 0, 0, 0]], dtype=torch.bool)
    xb = i["x"] * i["B"][:, :, 0]
    want = torch.cat([xb[:, :3].cumsum(1), xb[:, 3:].cumsum(1)], 1) * i["C"][:, :, 0]
    assert torch.allclose(D.scan(i)["y"][0], want, rtol=0, atol=1e-14)
