"""The gate's sigmoid over its whole range, where a far gate leaves little of the block.

Without norms do = scale sigmoid(gate) dr_out. u = 2^-24: the exponential is
within one step (2 u), the sum with 1 and the quotient round once each, and three
products remain at most: 7 u, taken as 8. Gates stay within 80, where sigmoid is a normal
number (1.8e-35)."""
import pytest

from test_block_norm import DT, EPS, U, lib_m

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["token", "full"])
def test_far_gates(kind, dt):
    M = lib_m()
    T, H = 320, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    gate = torch.linspace(-80, 80, T, device="cuda")
    if kind == "full":
        gate = (gate[:, None] + torch.rand(T, H, generator=g, device="cuda") - 0.5).clamp(-80, 80).to(DT[dt])
    d = (1 + torch.rand(T, H, generator=g, device="cuda")).to(DT[dt])
    o = torch.randn(T, H, generator=g, device="cuda")
    do = torch.full((T, H), float("nan"), device="cuda")
    M.moe_block_norm_grad(o, None, M.MPB_BF16 if dt == "bf16" else M.MPB_F16, gate, None, None, 0.75, EPS, d, None,
                          torch.empty_like(d), do, None, None, None, None)
    g64 = gate.double() if kind == "full" else gate.double()[:, None]
    want = 0.75 * d.double() / (1 + torch.exp(-g64))
    rel = ((do.double() - want).abs() / want).amax(1)
    assert float(rel.max()) <= 8 * U, f"{float(rel.max() / U):.1f} u at gate {float(gate[rel.argmax()].double().mean()):.1f}"
