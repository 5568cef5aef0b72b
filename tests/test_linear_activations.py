"""The activations of moe_linear and their derivatives where their accuracy shows: results of 16 bits next to a residual
that cancels them, and far out.

Tolerances, u = 2^-24, from the operations of each form. Results of 16 bits. A sigmoid is one exponential and one
reciprocal: within (6 + |x|) u of itself, so z sigmoid(x) with x = z or x = 2 sqrt(2 / pi) (z + 0.044715 z^3), which
is itself within 4 u, within (8 + 5 |x|) u. gelu is z (1 - tail) or z tail, tail = Phi(-|z|) by an exponential and a
polynomial: the fit 2^-25, the polynomial's argument 3 u times a condition of 3, its own additions 3 u, exponential and
products 4 u, the exponential's argument z^2 u: tail within (18 + 1.1 z^2) u of itself. fp32 results: a sigmoid within
6 u, erfc within 8 u and its argument within 2 u of itself."""
import math

import pytest

import test_linear as TL
from test_linear import ACTS, DT, U

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def through_the_bias(z, act, t, res=None):
    """moe_linear of zeros with bias z: (y of type t, the stored z)."""
    M = TL.lib_m()
    N, xt = z.shape[0], torch.float16 if t is torch.float32 else t
    X, W = torch.zeros(1, 64, dtype=xt, device="cuda"), torch.zeros(N, 64, dtype=xt, device="cuda")
    y, zs = torch.empty(1, N, dtype=t, device="cuda"), torch.empty(1, N, dtype=xt, device="cuda")
    ws = torch.empty(M.moe_linear_workspace_bytes(1, 64, N), dtype=torch.uint8, device="cuda")
    M.moe_linear(X, M.MPB_BF16 if xt is torch.bfloat16 else M.MPB_F16, W, z, ACTS.index(act), res, zs, y, ws)
    return y[0], zs[0]


def off16(z, a, act):
    """What act of 16-bit results may be off before it is rounded."""
    if act in ("none", "relu"):
        return torch.zeros_like(z)
    if act == "gelu":
        tail = 0.5 * torch.special.erfc(z.abs() / math.sqrt(2))
        return 1.05 * z.abs() * tail * (18 + 1.1 * z * z) * U + 3 * U * a.abs()
    x = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(-x)  # the exponent's error does not reach a sigmoid near 1
    return 1.05 * (8 + 5 * x.abs() * s) * U * a.abs()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_next_to_a_residual_that_cancels(dt, act):
    """y = res + act(z) with res the nearest 16-bit value to -act(z): what is left shows act's own error."""
    t = DT[dt]
    z = torch.linspace(-6, 6, 20000, device="cuda")
    zd = z.double().cpu()
    a, _ = TL.act64(zd, act)
    res = (-a).to(t)
    y, _ = through_the_bias(z, act, t, res.cuda()[None])
    ref = a + res.double()
    tol = off16(zd, a, act) + U * ref.abs()
    TL.check(y.cpu(), ref, tol + 1.01 * TL.half_step(t, ref.abs() + tol), act)
