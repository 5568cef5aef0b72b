"""Operands that the entries take in any alignment, at odd addresses; a router without bias; and gradients of routing
weights that hold anything where a slot does not count."""
import pytest

import test_adapters as TA
import test_block_norm as TN
import test_router_loss as TR

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def shifted(v):
    """The same values one element behind an aligned address."""
    if v is None:
        return None
    w = torch.empty(v.numel() + 1, dtype=v.dtype, device=v.device)[1:].view(v.shape)
    return w.copy_(v)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_odd_addresses(dt):
    d = TA.inputs(300, 128, 192, 3, 24, dt, seed=1)
    want = TA.run(d, dt)
    assert torch.equal(TA.run({**d, **{k: shifted(d[k]) for k in ("ranks", "scales", "adapter")}}, dt), want)
    small = {k: v[:40].contiguous() if k in ("X", "adapter", "base") else v for k, v in d.items()}
    want = TA.run(small, dt)
    assert torch.equal(TA.run({**small, **{k: shifted(small[k]) for k in ("ranks", "scales", "adapter")}}, dt), want)

    d = TN.inputs(70, 320, dt, "token", True, True, seed=2)
    e = {**d, "gate": shifted(d["gate"])}
    for a, b in zip(TN.run_fwd(d, dt, 0.7), TN.run_fwd(e, dt, 0.7)):
        assert torch.equal(a, b)
    a, b = TN.run_grad(d, dt, 0.7), TN.run_grad(e, dt, 0.7)
    assert all(torch.equal(a[k], b[k]) for k in a)

    d = TR.inputs(130, 192, 12, 3, dt, True, seed=3)
    e = {**d, **{k: shifted(d[k]) for k in ("b", "idx", "mask", "gw")}}
    o = TR.run_fwd(d, dt)
    p = TR.run_fwd(e, dt)
    assert all(torch.equal(o[k], p[k]) for k in o)
    a, b = TR.run_grad(d, dt, o), TR.run_grad(e, dt, {k: shifted(v) for k, v in o.items()})
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("T,H,E,K", [(1, 128, 16, 16), (333, 256, 60, 4), (8200, 128, 130, 5)])
def test_no_bias(T, H, E, K):
    d = TR.inputs(T, H, E, K, "f16", T > 1, bias=False, seed=4)
    o = TR.run_fwd(d, "f16")
    TR.check_fwd(d, "f16", o)
    TR.check_grad(d, "f16", TR.run_grad(d, "f16", o))


def test_weight_gradients_of_slots_that_do_not_count():
    """gw of masked tokens and of ids out of range may hold nan: the same bits as with zeros there."""
    d = TR.inputs(140, 128, 16, 4, "bf16", True, seed=5)
    d["idx"][::7, 1] = 16
    d["idx"][::5, 2] = -3
    out = (d["idx"] < 0) | (d["idx"] >= 16) | (d["mask"] == 0)[:, None]
    assert int(out.sum()) > 50
    o = TR.run_fwd(d, "bf16")
    a = TR.run_grad({**d, "gw": d["gw"].masked_fill(out, 0.0)}, "bf16", o)
    b = TR.run_grad({**d, "gw": d["gw"].masked_fill(out, float("nan"))}, "bf16", o)
    for k in a:
        assert torch.isfinite(a[k]).all() and torch.equal(a[k], b[k]), k
