"""dX of moe_linear_grad where dz is not dy itself (an activation, or fp32 dy): as exact as dz in fp32 makes it.

Tolerances. u = 2^-24. dz in two fp16 parts is within 2^-22 of itself and 2^-38 of the largest |dy|, its own fp32
error within 32 u (1 + |z|) |dy| + u |dz| (0 for fp32 dy taken as it is), bf16 W within 2^-38 of its largest. The
reduction runs over both parts, 2 N terms: E(2 N) = (2 N / 32 + 64) u of their absolute sum. The result's rounding
adds half a step. A part of 11 bits is off by up to 2^-12 of each term: where a sum cancels, that is many half steps."""
import pytest

import linear_plans
import test_linear as TL
from test_linear import DT, U, E

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def reference(d, dt, dy, act):
    """(dX in 64 bits, what each element may be off before it is rounded)."""
    W, z, dy = d["W"].double(), d["z"].double(), dy.double()
    dz = dy * (TL.act64(z, act)[1] if act != "none" else 1)
    own = (32 * U * (1 + z.abs()) * dy.abs() + U * dz.abs()) if act != "none" else 0
    off = own + (1.01 * 2.0 ** -22 + E(2 * W.shape[0])) * dz.abs() + 2.0 ** -38 * dy.abs().max()
    w_off = 2.0 ** -38 * W.abs().max() if dt == "bf16" else 0.0
    return dz @ W, off @ W.abs() + w_off * dz.abs().sum(1)[:, None]


# stages that end at the reduction's end and inside it, in the middle of the two parts; split reductions; each tile
SHAPES = [(40, 128, 8, 128), (300, 256, 72, 128), (500, 512, 264, 128), (4001, 2816, 72, 192), (4088, 4096, 72, 256),
          (4093, 4096, 64, 256)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act,dyt", [("none", "f32"), ("silu", "16"), ("gelu", "f32")])
@pytest.mark.parametrize("T,Kd,N,rows", SHAPES)
def test_input_gradient_keeps_dz_s_bits(T, Kd, N, rows, act, dyt, dt):
    assert linear_plans.plan(T, Kd, N, 2)[0] == rows
    d = TL.inputs(T, Kd, N, dt, seed=21)
    dy = TL.gradient_of(T, N, dt if dyt == "16" else "f32", d["g"], 1.0)
    ref, off = reference(d, dt, dy, act)
    for want in (("dX",), ("dX", "dW", "db")):  # alone, and in one launch with dW where tiles are small
        out = TL.run_grad(d, dt, dy, act, want=want)["dX"]
        TL.check(out, ref, off + 1.01 * TL.half_step(DT[dt], ref.abs() + off), "dX")


def test_input_gradient_of_a_split_reduction():
    assert linear_plans.plan(40, 128, 2048, 2)[1] > 1
    d = TL.inputs(40, 128, 2048, "f16", seed=22)
    dy = TL.gradient_of(40, 2048, "f32", d["g"], 1.0)
    ref, off = reference(d, "f16", dy, "none")
    out = TL.run_grad(d, "f16", dy, "none", want=("dX",))["dX"]
    TL.check(out, ref, off + 1.01 * TL.half_step(torch.float16, ref.abs() + off), "dX")


@pytest.mark.parametrize("act,dyt", [("none", "f32"), ("silu", "f16")])
def test_norm_of_the_error_is_that_of_the_rounding(act, dyt):
    """512 tokens of 2048 x 512 in fp16: dX is off by as much as the exact result rounded, 2.1e-4 of its norm. What
    is added before the rounding has at most 2^-21 of the terms' norm, 1e-5 of the result's for sums of random
    signs; a tenth of the rounding's 2.1e-4 would add half a percent, the sample of 262144 elements 0.2. 11 bits of
    dz make it 2.9e-4."""
    d = TL.inputs(512, 512, 2048, "f16", seed=23)
    dy = TL.gradient_of(512, 2048, dyt, d["g"], 1.0)
    ref, _ = reference(d, "f16", dy, act)
    got = TL.run_grad(d, "f16", dy, act, want=("dX",))["dX"].double()
    assert float((got - ref).norm()) <= 1.02 * float((ref.half().double() - ref).norm())


@pytest.mark.parametrize("dyt", ["f16", "f32"])
def test_infinite_gradients_keep_their_sign(dyt):
    """An infinite dz has nothing left for its second part: sums are infinite, of the formula's sign, not nan."""
    d = TL.inputs(70, 128, 72, "f16", seed=24)
    dy = TL.gradient_of(70, 72, dyt, d["g"]).clone()
    dy[3, 5], dy[9, 7], d["z"][3, 5], d["z"][9, 7] = float("inf"), -float("inf"), 1.0, 1.0
    d["X"][d["X"] == 0], d["W"][d["W"] == 0] = 1.0, 1.0
    out = TL.run_grad(d, "f16", dy, "silu")
    W, X = d["W"].double(), d["X"].double()
    assert torch.equal(out["dX"][3].double(), float("inf") * W[5]) and torch.equal(out["dX"][9].double(), -float("inf") * W[7])
    assert torch.equal(out["dW"][5].double(), float("inf") * X[3]) and torch.equal(out["dW"][7].double(), -float("inf") * X[9])


@pytest.mark.parametrize("T,Kd,N", [(70, 128, 264), (4001, 2816, 72)])
@pytest.mark.parametrize("up", [122, -100])
def test_scales_far_apart(up, T, Kd, N):
    """Gradients near one end of bf16's range with operands that bring the products back: no overflow on the way."""
    d = TL.inputs(T, Kd, N, "bf16", seed=25)
    other = 2.0 ** (-60 if up > 0 else 60)
    d["X"] *= other
    d["W"] *= other
    dy = TL.gradient_of(T, N, "bf16", d["g"]) * 2.0 ** up  # of 0.1: the largest is near 2^(up - 1)
    out = TL.run_grad(d, "bf16", dy, "silu", want=("dX", "dW"))
    assert out["dX"].isfinite().all() and out["dW"].isfinite().all()
    TL.check_grad(d, "bf16", dy, "silu", out)
