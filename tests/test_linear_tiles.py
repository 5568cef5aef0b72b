"""moe_linear and moe_linear_grad through every kernel that the rule of sizes can choose: each test first asserts that
its sizes take the kernel that it is there for. Tolerances as derived in test_linear."""
import pytest

import linear_plans
import test_linear as TL

torch = pytest.importorskip("torch")


def few(T, Kd, N):
    """linear_skinny: up to 128 tokens whose repeated reading costs less than a join."""
    return T <= 128 and (T - 1) * N * Kd <= 270000000


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T", [32, 33, 48, 49, 64, 65, 80, 81, 96, 97, 112, 113, 128])
def test_few_tokens_of_every_count_of_rows(T, dt):
    """16 tokens a matrix instruction, 1 to 8 of them; reductions of 20 pieces for 16 waves; columns inside a group of 16."""
    Kd, N = 1280, 72
    assert few(T, Kd, N)
    d = TL.inputs(T, Kd, N, dt, res=dt, seed=31)
    TL.check_fwd(d, dt, dt, "silu", *TL.run_fwd(d, dt, dt, "silu"))
    d["res"] = None
    TL.check_fwd(d, dt, "f32", "none", *TL.run_fwd(d, dt, "f32", keep=False))


# tokens, reduction, columns, rows of a tile; edges inside a tile in both directions
FORWARD = [(4093, 192, 5632, 192), (4001, 64, 2824, 192), (3001, 64, 4104, 256), (150, 64, 1000, 128)]


def test_forward_tiles_are_those_meant():
    for T, Kd, N, rows in FORWARD:
        assert linear_plans.plan(T, N, Kd)[0] == rows and not few(T, Kd, N)
    assert {rows for *_, rows in FORWARD} == {128, 192, 256}


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "gelu"])
@pytest.mark.parametrize("dt,y", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("T,Kd,N,rows", FORWARD)
def test_forward_tiles(T, Kd, N, rows, dt, y, act):
    d = TL.inputs(T, Kd, N, dt, res=y, seed=32)
    a = TL.run_fwd(d, dt, y, act)
    TL.check_fwd(d, dt, y, act, *a)
    b = TL.run_fwd(d, dt, y, act, in_place=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# T, Kd, N, rows of dX's tile and of dW's, with one part of dz and with two
GRADIENTS = [(1025, 4096, 4088, (128, 256), (128, 256)), (4001, 2816, 264, (192, 128), (192, 128)),
             (4093, 4096, 72, (256, 128), (256, 128)), (1025, 2816, 4088, (128, 192), (128, 192)),
             (300, 320, 264, (128, 128), (128, 128))]


def test_gradients_tiles_are_those_meant():
    plans = [((linear_plans.plan(T, Kd, N, parts)[0], linear_plans.plan(N, Kd, T, parts)[0]), given)
             for T, Kd, N, *both in GRADIENTS for parts, given in zip((1, 2), both)]
    assert all(a == b for a, b in plans), plans
    for i in (0, 1):
        assert {b[i] for _, b in plans} == {128, 192, 256}


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,Kd,N", [g[:3] for g in GRADIENTS])
def test_gradients_tiles(T, Kd, N, dt, act):
    d = TL.inputs(T, Kd, N, dt, seed=33)
    dy = TL.gradient_of(T, N, dt, d["g"])
    out = TL.run_grad(d, dt, dy, act)
    TL.check_grad(d, dt, dy, act, out)
    for k in ("dX", "dW"):  # alone, where a launch of both is not made
        assert torch.equal(TL.run_grad(d, dt, dy, act, want=(k,))[k], out[k])
