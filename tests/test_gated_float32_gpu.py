"""How exact the activations of float32 are, against 64-bit values at the products
that the call itself gives: applied to the sums as they leave the tensor cores (the
special function unit's exponential and reciprocal) and to products in memory (expf,
erfcf and a division), forward and backward.

Tolerances in units e = 2^-23, from the documented errors of what is called: __expf(x)
2 + 1.2 |x|, the approximate reciprocal 1 and quotient 2, expf 1, erfcf 4; any other
operation rounds by e / 2.
  An exponent that is itself rounded adds its absolute error: 3 |q| for gelu_tanh's q
(six roundings), a / 2 for gelu's a = g^2 / 2.
  Special function unit: s = 1 / (1 + exp(-q)) 3.5 + 1.2 |q|, times g 4 + 1.2 |q|.
gelu's tail is exp(-a) t poly(t): 2 + 1.7 a for the exponential, 3 for t, which the
product passes on 3.5 times at most, 3 for the polynomial's roundings and 1 for its
fit, 2 for the products and 1 for those with g: below 23 + 1.7 a.
  Exactly: s 3 (its smaller half is exp's times the larger), times g 3.5; erfcf's
argument is off by 1.1, which erfc passes on g^2 + 1 times: 6 + 1.1 g^2.  The slopes
are sums of two such terms: see `slope_of`.
  Results below 2^-121 may be 0, since exp(88.8) is infinite."""
import numpy as np
import pytest

from tests.test_gated_gpu import ACTS, act64, close
from tests.test_product_gpu import mods

pytestmark = pytest.mark.gpu

E = 2.0 ** -23
C = (8 / np.pi) ** 0.5


def q_of(act, g):
    return C * (g + 0.044715 * g ** 3) if act == "gelu_tanh" else g


def units(act, g, approximate):
    """Of the activation's relative error."""
    q, a = q_of(act, g).abs(), g * g / 2
    if act == "relu":
        return 0 * g
    if approximate:
        return 23 + 1.7 * a if act == "gelu" else 4 + 1.2 * q + (3 * q if act == "gelu_tanh" else 0)
    return 6 + 2.2 * a if act == "gelu" else 3.5 + (3 * q if act == "gelu_tanh" else 0)


def slope_of(act, g):
    """The slope, and its error in units of 1."""
    torch, _ = mods()
    _, slope = act64(act, g)
    q, a = q_of(act, g), g * g / 2
    if act == "relu":
        return slope, 0 * g
    if act == "gelu":
        density, p = torch.exp(-a) / (2 * np.pi) ** 0.5, 0.5 * torch.special.erfc(-g / 2 ** 0.5)
        err = (2 + 0.5 * a) * g.abs() * density + (6 + 2.2 * a) * p
    else:
        s, off = torch.sigmoid(q), (3 * q.abs() if act == "gelu_tanh" else 0)
        rest = s * torch.sigmoid(-q)
        if act == "sigmoid":
            # (1 - s is 0 in 64 bits from g = 37 on, where it is 9e-17; s(-g) is not)
            return rest, 5 * rest * E
        dq = C * (1 + 0.134145 * g ** 2) if act == "gelu_tanh" else 1
        err = (8 + off) * g.abs() * dq * rest + (3 + off) * s
    return slope, torch.nan_to_num(err + 0.5 * slope.abs()) * E


def values(rows):
    """rows x 32 of g: close together around 0, in both tails and far away."""
    torch, _ = mods()
    far = [0.0, 1e-30, -1e-30, 1e-6, -1e-6, 20.0, -20.0, 50.0, -50.0, 80.0, -80.0, 86.0, -86.0, 88.0, -88.0, 89.0, -89.0, 300.0, -300.0, 6e4, -6e4, 1e30, -1e30]
    near = np.linspace(-14, 14, 126 * 32 - len(far))
    g = torch.tensor(np.concatenate([far, near]), dtype=torch.float32, device="cuda").reshape(126, 32)
    return g.repeat((rows + 125) // 126, 1)[:rows].contiguous()


# in the drain; by the sums of a cluster; products in memory, then a pass
@pytest.mark.parametrize("rows,k,approximate", ((126, 64, True), (126, 520, True), (8448, 520, False)))
@pytest.mark.parametrize("act", ACTS)
def test_activations_forward(act, rows, k, approximate):
    torch, sr = mods()
    g = values(rows)
    u = torch.linspace(-2, 2, 32, device="cuda").expand(rows, 32)
    x = torch.zeros(rows, k, device="cuda")
    x[:, :32], x[:, 32:64] = g, u
    w = torch.zeros(1, k, 64, device="cuda")
    w[0, :64] = torch.eye(64, device="cuda")
    off = torch.tensor([0, rows], device="cuda")
    out, pre = sr.seg_gated(x, w, off, act, with_pre=True)
    close(pre, x[:, :64].double(), 2.0 ** -20 * x[:, :64].double().abs(), (act, "pre"))
    assert torch.equal(out, sr.seg_gated(x, w, off, act))
    gate, other = pre[:, :32].double(), pre[:, 32:].double()
    want = torch.nan_to_num(act64(act, gate)[0]) * other
    close(out, want, units(act, gate, approximate) * E * want.abs() + 2.0 ** -121 * other.abs(), (act, rows, k))


@pytest.mark.parametrize("act", ACTS)
def test_activations_backward(act):
    """The gradient of the products, before the products with it."""
    torch, sr = mods()
    top = torch.finfo(torch.float32).max
    g = values(126)
    g[0, 0], g[0, 1] = top, -top
    u = torch.linspace(-2, 2, 32, device="cuda").expand(126, 32).contiguous()
    dy = torch.linspace(0.5, 1.5, 126, device="cuda")[:, None].expand(126, 32).contiguous()
    pre, dpre = torch.cat([g, u], dim=1), torch.empty(126, 64, device="cuda")
    code = sr.load_library().seg_gated_grad(pre.data_ptr(), sr.SEG_F32, 126, 32, 64, dy.data_ptr(), sr.SEG_F32, 32, sr.ACTIVATIONS[act],
                                            dpre.data_ptr(), 64, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    gate, d = g.double(), dy.double()
    f = torch.nan_to_num(act64(act, gate)[0])
    slope, err = slope_of(act, gate)
    slope = torch.nan_to_num(slope)
    both = (d * u.double()).abs()
    close(dpre[:, :32], d * u.double() * slope, both * (err + 0.5 * E * slope.abs()) + 2.0 ** -121 * both, (act, "slope"))
    close(dpre[:, 32:], d * f, d * f.abs() * units(act, gate, False) * E + 2.0 ** -121 * d, (act, "activation"))
