"""A residual block as it is used: norm, router, packed experts, adapters, norm
with gate and residual scale, then the router's losses and the backward pass,
each step held to its formula in 64 bits on the step's own inputs."""
import numpy as np
import pytest

import mpb_synth as S
import oracle as O
import test_adapters as TA
import test_block_norm as TN
import test_router_loss as TR
from helpers import assert_close

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def routed(D, L, x, xdtype):
    """The oracle's routing and expert output of activations x."""
    X = x.double().cpu().numpy()
    z, w, _ = O.route(X, L.W_r, L.bias, L.K)
    return z, w, O.moe_ffn(X, z, w, L)


@pytest.mark.parametrize("cfg,T", [(0, 16), (0, 1), (10, 72), (11, 9)])
def test_two_blocks_and_their_gradients(layer_cache, cfg, T):
    from mixed_precision_bit_amd import _lib as M
    from mixed_precision_bit_amd.layer import DeviceLayer
    L = layer_cache(cfg)
    D = DeviceLayer.from_synth(L)
    M.mpb_init(D.H, D.I, D.E, D.S, D.K, D.q_dev, L.q)
    xd = L.cfg["xdtype"]
    d = TN.inputs(T, D.H, xd, "token", True, True, seed=cfg)
    ad = TA.inputs(T, D.H, D.H, 3, 16, xd, seed=cfg)
    ad["adapter"][0] = 1
    r, x = d["r"], D.norm_in(d["r"], xd, d["gn"])
    TN.check_fwd({**d, "gate": None, "gp": None}, xd, 1.0, None, x, no_o=True)
    for step in range(2):
        idx, w, out, r_out, x_next = D.block(x, r, xd, d["gp"], d["gn"], d["gate"], 0.7, adapters=ad)
        plain = D.forward(x, xd)
        assert torch.equal(plain[0], idx) and torch.equal(plain[1], w)
        z, wo, ref = routed(D, L, x, xd)
        assert np.array_equal(idx.cpu().numpy(), z)
        assert_close(plain[2].cpu().numpy(), ref, f"experts {step}")
        TA.check({**ad, "X": x, "base": plain[2]}, out)
        here = {**d, "o": out, "r": r}
        TN.check_fwd(here, xd, 0.7, r_out, x_next)
        # backward of the norms, and the router's losses with a gradient of the weights
        g = D.block_norm_grad(out, r_out, xd, d["dr_out"], d["dx"], d["gp"], d["gn"], d["gate"], 0.7)
        TN.check_grad({**here, "r": r_out}, xd, 0.7, {"dr": g["r"], "do": g["out"], "dgate": g["gate"],
                                                      "dgp": g["gamma_post"], "dgn": g["gamma_next"]})
        s = D.router_loss(x, xd, idx)
        q = {"X": x, "W": D.W_r, "b": D.bias, "idx": idx, "mask": None, "gw": torch.randn_like(w)}
        TR.check_fwd(q, xd, s)
        dX, dW, db = D.router_loss_grad(s, gw=q["gw"])
        TR.check_grad(q, xd, {"dX": dX, "dW": dW, "db": db})
        mass = torch.empty(D.E, dtype=torch.float64, device="cuda")
        M.moe_routing_mass(idx, torch.ones_like(w), D.E, mass)
        assert torch.allclose(mass * s["counts"][D.E] * D.K, s["counts"][:D.E].double())  # the counts are the routing's
        r, x = r_out, x_next


def test_block_under_graph_replay(layer_cache):
    """The whole block captured on one stream and replayed on other inputs, eager work between the replays."""
    from mixed_precision_bit_amd import _lib as M
    from mixed_precision_bit_amd.layer import DeviceLayer
    L = layer_cache(0)
    D = DeviceLayer.from_synth(L)
    M.mpb_init(D.H, D.I, D.E, D.S, D.K, D.q_dev, L.q)
    sets, want = [], []
    for k in (1, 2):
        d, ad = TN.inputs(16, D.H, "f16", "full", True, True, seed=k), TA.inputs(16, D.H, D.H, 3, 8, "f16", seed=k)
        sets.append((d, ad))
        x = D.norm_in(d["r"], "f16", d["gn"])
        b = D.block(x, d["r"], "f16", d["gp"], d["gn"], d["gate"], 0.7, adapters=ad)
        want.append([t.clone() for t in (*b, *D.router_loss_grad(D.router_loss(x, "f16", b[0])))])
    d, ad = ({k: None if v is None else v.clone() for k, v in q.items()} for q in sets[0])
    D.alloc_route(16)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x = D.norm_in(d["r"], "f16", d["gn"])
        b = D.block(x, d["r"], "f16", d["gp"], d["gn"], d["gate"], 0.7, adapters=ad)
        got = (*b, *D.router_loss_grad(D.router_loss(x, "f16", b[0])))
    for k in (1, 0, 1, 0):
        for dst, src in ((d, sets[k][0]), (ad, sets[k][1])):
            for name, v in dst.items():
                if v is not None:
                    v.copy_(src[name])
        g.replay()
        torch.cuda.synchronize()
        for a, c in zip(got, want[k]):
            assert torch.equal(a, c)
        D.forward(x, "f16")


def test_block_on_its_own_stream(layer_cache):
    """Everything on a stream other than the current one, the current one writing into fresh memory meanwhile."""
    from mixed_precision_bit_amd import _lib as M
    from mixed_precision_bit_amd.layer import DeviceLayer
    L = layer_cache(0)
    D = DeviceLayer.from_synth(L)
    d, ad = TN.inputs(16, D.H, "f16", "token", True, True, seed=3), TA.inputs(16, D.H, D.H, 3, 8, "f16", seed=3)
    mask = torch.arange(16, device="cuda") % 5 != 0  # a bool mask

    def all_of(stream):
        x = D.norm_in(d["r"], "f16", d["gn"], stream=stream)
        b = D.block(x, d["r"], "f16", d["gp"], d["gn"], d["gate"], 0.7, adapters=ad, stream=stream)
        g = D.block_norm_grad(b[2], b[3], "f16", d["dr_out"], d["dx"], d["gp"], d["gn"], d["gate"], 0.7, stream=stream)
        s = D.router_loss(x, "f16", b[0], mask, stream=stream)
        return [*b, *g.values(), s["loss"], s["counts"], *D.router_loss_grad(s, stream=stream)]

    M.mpb_init(D.H, D.I, D.E, D.S, D.K, D.q_dev, L.q)
    want = all_of(None)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    M.mpb_init(D.H, D.I, D.E, D.S, D.K, D.q_dev, L.q, stream=st)
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = all_of(st)
        junk = [torch.full((1 << 18,), float("nan"), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        for a, c in zip(got, want):
            assert torch.equal(a, c)
    M.mpb_init(D.H, D.I, D.E, D.S, D.K, D.q_dev, L.q)
