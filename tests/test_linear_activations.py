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


FAR = [0.0, -0.0, 1e-30, -1e-30, 0.5, -0.5, 6, -6, 11, -11, 13, -13, 19.9, -19.9, 20.1, -20.1, 30, -30, 88, -88, 90, -90, 119, -119, 121, -121,
       3e4, -3e4, 6.5e4, -6.5e4]
FARTHER = [1e18, -1e18, 1e30, -1e30, 3e38, -3e38]  # past fp16's range


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_far_out(act, dt):
    """Values up to bf16's largest and infinities. Results below 2^-126, fp32's smallest normal number, may be 0, and a
    sigmoid under 2^-128 with them: |z| 2^-125 for |z| up to 121."""
    t = DT[dt]
    z = FAR + FARTHER + [float("inf"), -float("inf")]
    z = torch.tensor([0.0] * (-len(z) % 8) + z, device="cuda")
    y = through_the_bias(z, act, t)[0].double().cpu()
    zd = z[:-2].double().cpu()
    a, _ = TL.act64(zd, act)
    a = torch.where(a.isnan(), 0.0, a)  # -z times e^inf in this formula's 64 bits
    tol = off16(zd, a, act).nan_to_num(0.0) + (16 * U * a.abs() if dt == "f32" else 0) + zd.abs().clamp(max=121) * 2.0 ** -125
    ref, got = a, y[:-2]
    over = ref.abs() >= torch.finfo(t).max  # rounds to infinity
    assert torch.equal(got[over], torch.full_like(got[over], float("inf")).copysign(ref[over]))
    TL.check(got[~over], ref[~over], (tol + (0 if dt == "f32" else 1.01 * TL.half_step(t, ref.abs() + tol)))[~over], act)
    assert y[-2] == float("inf")
    assert y[-1] == -float("inf") if act == "none" else y[-1] == 0 if act == "relu" else y[-1].isnan() or y[-1] == 0  # -inf times 0


@pytest.mark.parametrize("dyt", ["16", "f32"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_gradients_far_out(act, dt, dyt):
    """dz = act'(z) for stored z far out and infinite: 0 or 1 there, and never nan. dX = dz through W = 1, dbias = dz."""
    t, M = DT[dt], TL.lib_m()
    z = torch.tensor(FAR + (FARTHER if dt == "bf16" else []) + [float("inf"), -float("inf")], device="cuda").to(t)
    z = torch.cat([z, torch.linspace(-25, 25, 512 - z.numel(), device="cuda").to(t)])[None]
    N = Kd = 512
    dy = torch.ones(1, N, device="cuda", dtype=torch.float32 if dyt == "f32" else t)
    X, W = torch.ones(1, Kd, device="cuda", dtype=t), torch.eye(N, device="cuda", dtype=t)
    dX, dW, db = torch.empty(1, Kd, device="cuda", dtype=t), torch.empty(N, Kd, device="cuda"), torch.empty(N, device="cuda")
    xt = TL.xd(dt)
    ws = torch.empty(M.moe_linear_grad_workspace_bytes(1, Kd, N, ACTS.index(act), TL.xd("f32") if dyt == "f32" else xt), dtype=torch.uint8, device="cuda")
    M.moe_linear_grad(X, xt, W, ACTS.index(act), z, dy, dX, dW, db, ws)
    x = z[0].double().clamp(-100, 100)  # beyond, the derivative is 0 or 1 to 64 bits
    ref = TL.act64(x, act)[1]
    # the sum of two terms, each within 32 u of itself, of which the second is at most |z| / 2 (see test_linear); an
    # exponential below 2^-126, fp32's smallest normal number, is 0, and is taken 1 + |z| times
    tol = 32 * U * (1 + x.abs().clamp(max=20)) * torch.where(x.abs() > 20, ref.abs(), 1.0) + (1 + x.abs()) * 2.0 ** -126
    TL.check(db, ref, tol, "dbias")
    tol = tol + 1.01 * 2.0 ** -22 * ref.abs() + 2.0 ** -38
    TL.check(dW, ref[:, None].expand(N, Kd), tol[:, None].expand(N, Kd), "dW")
    TL.check(dX[0], ref, tol + 1.01 * TL.half_step(t, ref.abs() + tol), "dX")
